"""Small pools for the tests of the decode-step operators: a layout, a pool
tensor with a guard behind it, and views of the pages of one layer.  The views
come from the layout's own queries (hkv_layer_info_get)."""
import numpy as np
import torch

import retrieve_store_chunk_amd as hkv
import workloads as W

TYPES = {"bf16": (torch.bfloat16, hkv.HKV_BF16), "fp16": (torch.float16, hkv.HKV_FP16),
         "fp32": (torch.float32, hkv.HKV_FP32), "e4m3": (torch.float8_e4m3fn, hkv.HKV_E4M3)}


def half_step(dtype) -> float:
    """The most one rounding to `dtype` is off, relative to the value."""
    return torch.finfo(dtype).eps / 2


class Pool:
    def __init__(self, path=0, blocks=8, block_size=0, mla_width=576, mla_bytes=2, heads=1,
                 head_dim=16, conv_bytes=2, conv_kernel=4, is_mla=(0, 1, 0, 1, 1), device="cuda",
                 conv_dim=None):
        desc = W._desc(list(is_mla), heads, head_dim,
                       3 * heads * head_dim if conv_dim is None else conv_dim, mla_bytes, path, 1,
                       block_size=block_size, mla_width=mla_width, conv_bytes=conv_bytes,
                       conv_kernel=conv_kernel)
        desc["pool_bytes"] = 1 << 34
        info = hkv.Layout(desc).info
        per_block = (info["n_slabs"] * info["unified_page_bytes"] if path == 0
                     else info["block_stride"])
        desc["pool_bytes"] = blocks * per_block
        self.layout = hkv.Layout(desc)
        self.desc, self.info, self.layers = desc, self.layout.info, self.layout.layers
        self.n = self.info["block_size"]
        self.blocks = self.info["num_blocks"]
        assert self.blocks == blocks
        used = self.info["pool_bytes_used"]
        self.bytes = torch.zeros(used, dtype=torch.uint8, device=device)
        self.mla = [i for i, m in enumerate(is_mla) if m]
        self.kda = [i for i, m in enumerate(is_mla) if not m]

    @property
    def ptr(self) -> int:
        return self.bytes.data_ptr()

    def rows(self, layer: int, dtype) -> torch.Tensor:
        """[blocks][N][width] view of an MLA layer's pages."""
        L, es, w = self.layers[layer], dtype.itemsize, self.desc["mla_width"]
        return self.bytes.view(dtype).as_strided(
            (self.blocks, self.n, w), (L["stride"] // es, w, 1), L["pool_offset"] // es)


def stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def tables(lens, n, blocks, rng, columns=None):
    """[seqs][columns] distinct shuffled block ids, 0x7FFFFFFF past a sequence's
    end (never to be read)."""
    need = [-(-max(0, x) // n) for x in lens]
    assert sum(need) <= blocks
    columns = columns or max(1, max(need))
    table = np.full((len(lens), columns), 0x7FFFFFFF, np.int32)
    ids, at = rng.permutation(blocks).astype(np.int32), 0
    for s, k in enumerate(need):
        table[s, :k] = ids[at:at + k]
        at += k
    return table
