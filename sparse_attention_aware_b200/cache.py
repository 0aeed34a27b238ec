"""The paged KV cache as the library's entry points take it: four device
tensors in the layout of the C ABI (``sa_kv_cache``).

  * k, v       : bf16 ``[num_pages][Hkv][P][d]`` -- one (page, kv head) tile is
    contiguous (``P*d*2`` bytes);
  * page_table : int32 ``[B][max_pages_per_seq]`` (logical page -> physical page);
  * seq_lens   : int32 ``[B]``.
"""
from __future__ import annotations

import dataclasses

import torch


@dataclasses.dataclass
class PagedCache:
    k: torch.Tensor            # bf16 [num_pages][Hkv][P][d]
    v: torch.Tensor            # bf16 [num_pages][Hkv][P][d]
    page_table: torch.Tensor   # int32 [B][max_pages]
    seq_lens: torch.Tensor     # int32 [B]

    @property
    def batch(self) -> int:
        return int(self.page_table.shape[0])

    @property
    def num_kv_heads(self) -> int:
        return int(self.k.shape[1])

    @property
    def page_size(self) -> int:
        return int(self.k.shape[2])

    @property
    def head_dim(self) -> int:
        return int(self.k.shape[3])

    @property
    def max_pages(self) -> int:
        return int(self.page_table.shape[1])

    @property
    def num_pages(self) -> int:
        return int(self.k.shape[0])

    def with_v(self, v: torch.Tensor) -> "PagedCache":
        return PagedCache(self.k, v, self.page_table, self.seq_lens)

    def to(self, device) -> "PagedCache":
        return PagedCache(self.k.to(device), self.v.to(device),
                          self.page_table.to(device), self.seq_lens.to(device))


@dataclasses.dataclass
class PagedCache4:
    """A cache held in 4 bits (``sa_kv4_cache``): one record of ``d + 16``
    bytes per (page, kv head, token) -- 4-bit codes of key and value, and a bf16
    scale and zero for each half of either.  ``rope_append`` writes it,
    ``expand_kv4`` reads pages back, ``sparse_decode_attn`` attends over it."""
    kv: torch.Tensor           # uint8 [num_pages][Hkv][P][d + 16]
    page_table: torch.Tensor   # int32 [B][max_pages]
    seq_lens: torch.Tensor     # int32 [B]

    @property
    def batch(self) -> int:
        return int(self.page_table.shape[0])

    @property
    def num_kv_heads(self) -> int:
        return int(self.kv.shape[1])

    @property
    def page_size(self) -> int:
        return int(self.kv.shape[2])

    @property
    def head_dim(self) -> int:
        return int(self.kv.shape[3]) - 16

    @property
    def max_pages(self) -> int:
        return int(self.page_table.shape[1])

    @property
    def num_pages(self) -> int:
        return int(self.kv.shape[0])

    @staticmethod
    def empty(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, page_table: torch.Tensor,
              seq_lens: torch.Tensor) -> "PagedCache4":
        """A cache of zeros on ``page_table``'s device."""
        kv = torch.zeros((num_pages, num_kv_heads, page_size, head_dim + 16), dtype=torch.uint8,
                         device=page_table.device)
        return PagedCache4(kv, page_table, seq_lens)

    def to(self, device) -> "PagedCache4":
        return PagedCache4(self.kv.to(device), self.page_table.to(device), self.seq_lens.to(device))


@dataclasses.dataclass
class PagePool:
    """The free pages of a paged cache, as a stack on the device
    (``plan_append`` pops and pushes; entries ``[0, free_count)`` are valid)."""
    free_pages: torch.Tensor   # int32 [capacity]
    free_count: torch.Tensor   # int32 [1]
    num_pages: int
    page_size: int

    @staticmethod
    def full(num_pages: int, page_size: int, device) -> "PagePool":
        """Every page free; page 0 is handed out first."""
        return PagePool(torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
                        torch.tensor([num_pages], dtype=torch.int32, device=device), num_pages, page_size)
