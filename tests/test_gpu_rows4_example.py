"""The 4-bit decode loop of examples/rows4_decode.py, small: no status bit, and
the last output within bf16 rounding (half a step, 2^-8, of the largest value)
and f16 probabilities (2^-11) of attention over the unpacked rows."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_loop_over_4_bit_rows():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("rows4_decode", os.path.join(ROOT, "examples", "rows4_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    requests, layers, heads, steps = 3, 2, 5, 4
    error, status, weights = example.run(requests, layers, heads, tokens=900, k=70, hot=256, steps=steps)
    assert error <= 2.0 ** -8 + 2.0 ** -10
    assert not any(status)
    # every head spreads a weight of 1 a step
    total = weights.double().sum(2)
    assert torch.allclose(total, torch.full_like(total, heads * steps), rtol=1e-4)


def loop(programmatic):
    """Swap-in, attention, eviction and backup of two layers in turn, without a
    host wait between them: outputs, weights and the handle's state at the end."""
    from hierarchical_sparse_kv_request_gb300 import hisparse as H
    R, L, heads, k, D, tokens, steps = 4, 2, 16, 96, 320, 1500, 6
    g = torch.Generator(device="cuda").manual_seed(11)
    hs = H.HiSparse(R, L, H.ROW4_BYTES, k, D, host_to_device_ratio=6, host_capacity=[tokens + steps] * R)
    hs.set_programmatic_launch(programmatic)
    for l in range(L):
        for r in range(R):
            kv = torch.randn((tokens, H.ROW4_VALUES), generator=g, device="cuda").bfloat16()
            H.pack_rows(kv, torch.from_numpy(hs.host_rows(l, r)[:tokens]))
    seq = torch.full((R,), tokens, dtype=torch.int32, device="cuda")
    hs.prefill(seq)
    topk = [torch.stack([torch.randperm(tokens, generator=g, device="cuda")[:k] for _ in range(R)]).int().contiguous()
            for _ in range(L * steps)]
    q = torch.randn((L * steps, R, heads, H.ROW4_VALUES), generator=g, device="cuda").bfloat16()
    new = torch.randn((L * steps, R, H.ROW4_VALUES), generator=g, device="cuda").bfloat16()
    packed = torch.empty((L, R, H.ROW4_BYTES), dtype=torch.uint8, device="cuda")
    out = torch.empty((L * steps, R, heads, H.ROW4_LATENT), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((L, R, k), dtype=torch.int32, device="cuda")
    plan = torch.empty((R, k, 2), dtype=torch.int32, device="cuda")
    misses = torch.empty((R,), dtype=torch.int32, device="cuda")
    weights = torch.zeros((L, R, tokens + steps), device="cuda")
    space = torch.empty(H.attend_workspace_bytes(R, heads, k, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for n in range(L * steps):
        l = n % L
        hs.swap_in(l, topk[n], seq, ids[l], plan, misses)
        hs.attend(l, q[n], ids[l], out[n], 0.05, positions=topk[n], weights=weights[l], workspace=space)
        hs.evict(l, weights[l], seq, 40, keep_recent=16, want=misses)
        H.pack_rows(new[n], packed[l])
        if l == L - 1:
            hs.backup_layers(list(range(L)), packed, seq)
            seq += 1
    torch.cuda.synchronize()
    assert not any(int(s) for s in hs.status())
    state = [[x.copy() for x in hs.read_state(l)] for l in range(L)]
    hs.close()
    return out, weights, state


def test_launches_that_overlap_change_nothing():
    import __graft_entry__
    __graft_entry__.build()
    (out, weights, state), (out2, weights2, state2) = loop(False), loop(True)
    assert torch.equal(out, out2) and torch.equal(weights, weights2)
    for a, b in zip(state, state2):
        assert all((x == y).all() for x, y in zip(a, b))
