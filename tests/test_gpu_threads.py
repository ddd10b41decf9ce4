"""The calls that encode tensor maps, from host threads that have made no CUDA call before (no context
is current there yet): tree attention and accumulated weight over more than 32 rows, prompts, and a
history in 8 bits give the main thread's bits."""
from __future__ import annotations

import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda"


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(DEV)


def _calls():
    import query_conditioned_kv_gb300 as kvc
    g = torch.Generator().manual_seed(1)
    H, Hq, D, BS, ctx, T = 2, 8, 128, 16, 300, 40
    mb = -(-(ctx + T) // BS)
    n_slots, bt = mb * BS, i32(np.arange(mb)[None])
    k, v = (torch.randn(n_slots, H, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(T, Hq, D, generator=g).bfloat16().to(DEV)
    c, off, n = i32([ctx]), i32([0, T]), i32([ctx + T])
    vis, zero = i32(ctx + 1 + np.arange(T)), i32([0])
    k8 = torch.randint(0, 120, (4, H, BS, D), generator=g, dtype=torch.uint8).to(DEV)
    one, t8, n8 = torch.ones(4, H, device=DEV), i32([[2, 0, 1]]), i32([48])
    lse_in = torch.full((1, T, Hq), 9.0, device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)

    def new():
        return (torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.zeros(T, Hq, device=DEV))

    def tree(o, s):
        kvc.kvc_tree_attn(q, k, v, n_slots, bt, mb, c, off, None, 0, 1, T, T, H, Hq, D, BS, 0.09, o[0], o[1],
                          ws, stream=s)

    def prompt(o, s):
        kvc.kvc_prompt_attn(q, k, v, n_slots, bt, mb, c, off, 1, T, T, H, Hq, D, BS, 0.09, o[0], o[1], stream=s)

    def q8(o, s):
        kvc.kvc_q8_attn(q, k8, k8, one, one, 4, t8, 3, n8, k, v, n_slots, bt, mb, c, off, None, 0, 1, T, T, H, Hq,
                        D, BS, 0.09, o[0], o[1], ws, stream=s)

    def mass(o, s):
        kvc.kvc_attn_mass(q[None], lse_in, T, None, vis, off, T, T, k[None], n_slots, bt, mb, n, zero, 1, 1, H, Hq,
                          D, BS, 0.09, 1.0, o[0], ws, stream=s)

    def new_mass():
        return (torch.zeros(1, 1, H, mb * BS, device=DEV),)

    return {"tree": (tree, new), "prompt": (prompt, new), "q8": (q8, new), "mass": (mass, new_mass)}


@pytest.mark.parametrize("name", ["tree", "prompt", "q8", "mass"])
def test_a_thread_without_a_context(name):
    call, new = _calls()[name]
    want, got = new(), new()
    stream = torch.cuda.current_stream().cuda_stream
    call(want, stream)
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            call(got, stream)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(torch.equal(a, b) for a, b in zip(got, want))
