"""Inputs and comparisons shared by the KV-cache tests."""
import numpy as np
import torch

from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# half a step of each type, relative to the value
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def make_pools(rng, n_pages, kvh, d, spread=0.3):
    """Codes of normal values and scales of a spread of sizes."""
    k, v = (o.e4m3_encode(np.clip(rng.normal(size=(n_pages, 64, kvh, d)) * 100, -448, 448)) for _ in range(2))
    ks, vs = (np.exp(spread * rng.normal(size=(n_pages, kvh))).astype(np.float32) * np.float32(0.01) for _ in range(2))
    return k, v, ks, vs


def make_table(rng, lens, n_pages, width=None):
    """A shuffled block table for requests of these lengths; unused entries are -1."""
    blocks = [-(-int(n) // 64) for n in lens]
    order = rng.permutation(n_pages)[: sum(blocks)]
    t = np.full((len(lens), width or max(max(blocks), 1)), -1, np.int32)
    at = 0
    for r, c in enumerate(blocks):
        t[r, :c] = order[at:at + c]
        at += c
    return t


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def attend_tolerance(dtype, d, ref, info):
    """Elementwise bounds on out and lse (see the derivation in test_gpu_kv_attend.py)."""
    n = info["n"]
    es = (d / 16 + 4) * 2.0 ** -22 * info["S"] + 2.0 ** -22 * (info["smax"] + 8)
    ew = 2.0 ** -21 if dtype == "f32" else 2.0 ** -11
    el = (n / 16 + 8) * 2.0 ** -22
    floor = n * 2.0 ** -37 * info["top"] * 448
    out = (2 * es + ew + 2 * el)[..., None] * info["A"] + HALF_STEP[dtype] * np.abs(ref) + floor[..., None] + 1e-30
    if dtype == "f16":
        out = out + 2.0 ** -25  # half a step of its subnormals
    return out, es + el


def run_attend(cfg, q, pools, table, n_slots, rows, listed=None, want_lse=True, status=None, stream=None, out=None,
               workspace=None):
    k, v, ks, vs = pools
    top_k = 0 if listed is None else listed.shape[-1]
    ws = spin.kv_workspace(cfg, rows, top_k) if workspace is None else workspace
    ws.fill_(255)                      # the workspace needs no initialisation: NaN bits
    out = torch.full_like(q, float("nan")) if out is None else out
    lse = torch.full(q.shape[:3], float("nan"), device="cuda") if want_lse else None
    spin.kv_attend(cfg, q, k, v, ks, vs, table, n_slots, rows, listed, out, lse, ws, status, stream)
    return out, lse
