"""A decode loop over a cache held in 4 bits, on synthetic keys and queries.

Per step and layer: swap the top-k rows in, attend over them by slot id with
each token's attention weight accumulated, free the hot rows that have gathered
the least of it, pack the step's new row and back it up.  At the end the last
step's output is compared with attention over the same rows unpacked.

    python examples/rows4_decode.py [--requests 8 --tokens 8000 --steps 16 ...]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from hierarchical_sparse_kv_request_gb300 import hisparse as H  # noqa: E402


def top_k(step_gen, seq, k, cap):
    """int32 [R][k]: mostly recent tokens, the others anywhere."""
    R = seq.numel()
    score = torch.rand((R, cap), generator=step_gen, device="cuda")
    pos = torch.arange(cap, device="cuda")
    score = score + 0.6 * torch.exp((pos - seq[:, None]) / (2.0 * k))
    return score.masked_fill(pos >= seq[:, None], -1).topk(k, 1).indices.to(torch.int32)


def run(requests=8, layers=2, heads=32, tokens=8000, k=512, hot=1536, steps=16, seed=0):
    dtype, scale = torch.bfloat16, H.ROW4_VALUES ** -0.5
    g = torch.Generator(device="cuda").manual_seed(seed)
    cap = tokens + steps
    hs = H.HiSparse(requests, layers, H.ROW4_BYTES, k, hot, host_to_device_ratio=-(-cap // hot),
                    host_capacity=[cap] * requests)
    for layer in range(layers):              # the prefix, packed straight into pinned host memory
        for r in range(requests):
            kv = torch.randn((tokens, H.ROW4_VALUES), generator=g, device="cuda").to(dtype)
            H.pack_rows(kv, torch.from_numpy(hs.host_rows(layer, r)[:tokens]))
    seq = torch.full((requests,), tokens, dtype=torch.int32, device="cuda")
    hs.prefill(seq)

    ids = torch.empty((requests, k), dtype=torch.int32, device="cuda")
    plan = torch.empty((requests, k, 2), dtype=torch.int32, device="cuda")
    misses = torch.empty((requests,), dtype=torch.int32, device="cuda")
    freed = torch.empty((requests,), dtype=torch.int32, device="cuda")
    out = torch.empty((requests, heads, H.ROW4_LATENT), dtype=dtype, device="cuda")
    lse = torch.empty((requests, heads), device="cuda")
    weights = torch.zeros((layers, requests, cap), device="cuda")
    space = torch.empty(H.attend_workspace_bytes(requests, heads, k, True), dtype=torch.uint8, device="cuda")
    new = torch.empty((layers, requests, H.ROW4_BYTES), dtype=torch.uint8, device="cuda")
    for step in range(steps):
        missed = 0
        for layer in range(layers):
            topk = top_k(g, seq, k, cap)
            q = torch.randn((requests, heads, H.ROW4_VALUES), generator=g, device="cuda").to(dtype)
            hs.swap_in(layer, topk, seq, ids, plan, misses)
            hs.attend(layer, q, ids, out, scale, lse=lse, positions=topk, weights=weights[layer], workspace=space)
            missed += int(misses.sum())
            if layer == layers - 1 and step == steps - 1:
                error = compare(hs, layer, q, ids, out, scale)
            # as many free slots as the step has missed, for the next one
            hs.evict(layer, weights[layer], seq, k, keep_recent=64, want=misses, out_counts=freed)
            kv = torch.randn((requests, H.ROW4_VALUES), generator=g, device="cuda").to(dtype)
            H.pack_rows(kv, new[layer])
        hs.backup_layers(list(range(layers)), new, seq)
        seq += 1
        print("step %2d: %5d of %d rows swapped in, %d hot rows freed in the last layer"
              % (step, missed, layers * requests * k, int(freed.sum())))
    status = [int(s) for s in hs.status()]       # (the words go with the handle)
    hs.close()
    print("largest error of the last output, relative to its largest value: %.4f" % error)
    return error, status, weights


def compare(hs, layer, q, ids, out, scale):
    """Largest difference of `out` from attention over the unpacked rows, relative
    to the largest value of the latter."""
    R, k = ids.shape
    hot = hs.device_buffer(layer).view(torch.uint8).reshape(R, hs.D, H.ROW4_BYTES)
    rows = torch.stack([hot[r][ids[r].long()] for r in range(R)])
    kv = torch.empty((R * k, H.ROW4_VALUES), dtype=q.dtype, device="cuda")
    H.unpack_rows(rows.view(R * k, H.ROW4_BYTES), kv)
    kv = kv.view(R, k, H.ROW4_VALUES).double()
    p = torch.softmax(torch.einsum("rhd,rkd->rhk", q.double(), kv) * scale, 2)
    want = torch.einsum("rhk,rkd->rhd", p, kv[..., :H.ROW4_LATENT])
    return float((out.double() - want).abs().max() / want.abs().max())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, default in (("requests", 8), ("layers", 2), ("heads", 32), ("tokens", 8000), ("k", 512),
                          ("hot", 1536), ("steps", 16), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=default)
    run(**vars(ap.parse_args()))
