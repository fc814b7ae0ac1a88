"""Runs of the 8-bit entry points with every written buffer between guard
bytes, as canary_cases.py does for the others: run_all() returns their bytes,
whether the guards are intact and the device status.  Run as a script (with
CSA_DEBUG=1: the debug build) it saves them."""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import compressed_sparse_attention_09_b200 as csa  # noqa: E402
from canary_cases import DEV, TC, Padded, _finish, _pack  # noqa: E402
from compressed_sparse_attention_09_b200 import synth  # noqa: E402


def rows_case(n, w, block, seed, name, out):
    nb = -(-w // block) if block else 1
    x = synth.make_normal((n, w), TC, seed).to(DEV)
    b = {"codes": Padded((n + 9, w), torch.uint8), "scales": Padded((n + 9, nb), torch.uint8),
         "y": Padded((n, w), torch.float32)}
    slots = torch.randperm(n + 9, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32).to(DEV)
    csa.csa_quantize_f8(csa.CSA_BF16, x, w, n, w, block, slots, n + 9, b["codes"].t, w, b["scales"].t, nb)
    csa.csa_dequantize_f8(csa.CSA_F32, b["codes"].t, w, b["scales"].t, nb, n + 9, w, block, slots, n, b["y"].t, w)
    _finish(name, b, out)


def gemm_case(M, N, K, kind, seed, name, out):
    kb = -(-K // 128)
    x, w = synth.make_normal((M, K), TC, seed).to(DEV), synth.make_normal((N, K), TC, seed + 1).to(DEV)
    b = {"a": Padded((M, K), torch.uint8), "sa": Padded((M, kb), torch.uint8), "b": Padded((N, K), torch.uint8),
         "sb": Padded((-(-N // 128), kb), torch.uint8), "d": Padded((M, N), kind),
         "ws": Padded((csa.csa_gemm_f8_workspace_bytes(M, N, K),), torch.uint8)}
    csa.csa_quantize_f8(csa.CSA_BF16, x, K, M, K, 128, None, 0, b["a"].t, K, b["sa"].t, kb)
    csa.csa_quantize_weight_f8(csa.CSA_BF16, w, K, N, K, b["b"].t, K, b["sb"].t, kb)
    csa.csa_gemm_f8(csa.CSA_F32 if kind == torch.float32 else csa.CSA_BF16, b["a"].t, K, b["sa"].t, kb, b["b"].t, K,
                    b["sb"].t, kb, M, N, K, b["d"].t, N, b["ws"].t)
    _finish(name, b, out)


def decode_case(dims, B, pos0, cap, steps, seed, name, out):
    m = dims.m
    packed = _pack(dims, synth.make_weights(dims, seed))
    n = B * cap
    b = {"packed8": Padded((csa.csa_packed_weights_f8_bytes(dims),), torch.uint8, torch.zeros((), dtype=torch.uint8)),
         "Cq": Padded((B, cap, dims.c), torch.uint8), "Cs": Padded((B, cap), torch.uint8),
         "Kq": Padded((B, cap, dims.cI), torch.uint8), "Ks": Padded((B, cap), torch.float32),
         "ring": Padded((B, 2 * m, csa.csa_ring_row_elems(dims)), torch.bfloat16,
                        synth.make_normal((B, 2 * m, csa.csa_ring_row_elems(dims)), dims, seed + 3)),
         "clen": Padded((B,), torch.int32, torch.full((B,), pos0 // m, dtype=torch.int32)),
         "ws": Padded((csa.csa_decode_f8_workspace_bytes(dims, B, cap),), torch.uint8)}
    csa.csa_pack_weights_f8(dims, packed.t, b["packed8"].t)
    csa.csa_quantize_f8(csa.CSA_BF16, synth.make_normal((n, dims.c), dims, seed + 1).to(DEV), dims.c, n, dims.c, 0, None, 0,
                        b["Cq"].t, dims.c, b["Cs"].t, 1)
    csa.csa_quantize_keys_e4m3(synth.make_normal((n, dims.cI), dims, seed + 2).to(DEV), dims.cI, n, dims.cI, b["Kq"].t,
                               b["Ks"].t)
    for step in range(steps):
        h = synth.make_normal((B, dims.d), dims, seed + 100 + step).to(DEV)
        b[f"O{step}"] = Padded((B, dims.nh * dims.c), torch.bfloat16)
        b[f"idx{step}"] = Padded((B, dims.topk), torch.int32)
        csa.csa_decode_f8(dims, packed.t, b["packed8"].t, h, torch.full((B,), pos0 + step, dtype=torch.int32, device=DEV),
                          b["ring"].t, b["Cq"].t, b["Cs"].t, b["Kq"].t, b["Ks"].t, b["clen"].t, cap, B, b[f"O{step}"].t,
                          b[f"idx{step}"].t, b["ws"].t)
    _finish(name, b, out)


def prefill_case(dims, lens, seed, name, out):
    T = sum(lens)
    cu, cb = csa.cu_from_lengths(lens, dims.m)
    NB = int(cb[-1])
    codes = torch.zeros(NB, dims.c, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(NB, dtype=torch.uint8, device=DEV)
    csa.csa_quantize_f8(csa.CSA_BF16, synth.make_normal((NB, dims.c), dims, seed).to(DEV), dims.c, NB, dims.c, 0, None, 0, codes,
                        dims.c, scales, 1)
    idx = torch.full((T, dims.topk), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for t in range(n):
            a = min(t // dims.m, dims.topk)
            idx[int(cu[b]) + t, :a] = torch.arange(a, dtype=torch.int32)
    b = {"O": Padded((T, dims.nh * dims.c), torch.bfloat16),
         "ws": Padded((csa.csa_mqa_f8_workspace_bytes(dims, T),), torch.uint8)}
    csa.csa_sparse_mqa_f8(dims, synth.make_normal((T, dims.nh * dims.c), dims, seed + 1).to(DEV), dims.nh * dims.c, codes, scales,
                          idx.to(DEV), cu.to(DEV), cb.to(DEV), len(lens), T, NB, b["O"].t, b["ws"].t)
    _finish(name, b, out)


def run_all():
    out = {}
    rows_case(33, 512, 0, 1, "rows", out)
    rows_case(21, 272, 128, 2, "blocks", out)
    gemm_case(5, 200, 1024, torch.float32, 3, "gemm_few", out)
    gemm_case(200, 300, 400, torch.bfloat16, 4, "gemm_many", out)
    gemm_case(131, 301, 400, torch.bfloat16, 8, "gemm_odd", out)
    gemm_case(131, 301, 400, torch.float32, 9, "gemm_odd_f32", out)
    decode_case(TC, B=1, pos0=2045, cap=640, steps=5, seed=5, name="decode_1", out=out)
    decode_case(TC, B=6, pos0=30, cap=40, steps=3, seed=6, name="decode_6", out=out)
    prefill_case(TC, [90, 1, 57], 7, "prefill", out)
    return out


if __name__ == "__main__":
    np.savez(sys.argv[1], **run_all())
