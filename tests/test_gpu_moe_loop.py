"""The decode step's layer loop with its MoE sublayers computed: every boundary and
every sublayer output against the oracle on what the GPU fed it, and a CUDA-graph
replay of the whole step that equals the eager run bit for bit."""

import numpy as np
import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M
from mhc_residual_stream_b200.decode import DecodeLoop
from mhc_residual_stream_b200.moe import MoeConfig

from _parity import assert_bf16_close
from _sublayer import assert_within, experts_bound, f64, linear_bound

CFG = MoeConfig(experts=24, intermediate=136, top_k=3, shared=192, num_groups=4, top_groups=2, weight_scale=1.5)


def test_schedule_with_moe_sublayers():
    from mhc_residual_stream_b200 import build
    build.build()
    loop = DecodeLoop(rows=2, hidden=256, layers=3, device="cpu", pack_fn=False, moe=CFG)
    assert [st.kind for st in loop.steps] == ["first", "ffn", "moe", "attn", "ffn", "moe", "attn", "ffn", "moe", "final"]
    bare = DecodeLoop(rows=2, hidden=256, layers=3, top_k=3, device="cpu", pack_fn=False)
    assert loop.algorithmic_bytes() == bare.algorithmic_bytes()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 20])
def test_moe_loop_stage_wise_and_captured(rows):
    loop = DecodeLoop(rows=rows, hidden=512, layers=3, device="cuda:0", moe=CFG)
    m = loop.moe_sublayer
    for st in loop.steps:
        if st.kind == "moe":
            loop.run_step(st)
            torch.cuda.synchronize()
            assert m.device_status() == M.OK
            x, w = f64(loop.layer_input), st.moe
            ex, bd = linear_bound(x, f64(w.router), None, "none", None, torch.float32)
            assert_within(m.logits, ex, bd, "logits")
            ow, ids = O.moe_route(f64(m.logits), 3, f64(w.bias), "sigmoid", 4, 2, 2, True, 1.5)
            e2p, prow, off = O.moe_permute(ids, 24)
            assert np.array_equal(m.expert_ids.cpu().numpy(), ids) and np.array_equal(m.e2p.cpu().numpy(), e2p)
            assert np.allclose(f64(m.expert_weights), ow, rtol=1e-5, atol=0)
            ex, bd = experts_bound(x, f64(w.w13), f64(w.w2), prow, off)
            assert_within(m.gemm2_permuted, ex, bd, "experts")
            ex, bd = linear_bound(x, f64(w.shared13), None, "swiglu", None, torch.bfloat16)
            assert_within(m.shared_inner, ex, bd, "shared gate-up")
            ex, bd = linear_bound(f64(m.shared_inner), f64(w.shared2), None, "none", None, torch.bfloat16)
            assert_within(m.shared_output, ex, bd, "shared down")
            continue
        a, b = st.src, st.dst
        inp = {k: f64(getattr(loop, k)[a]) for k in ("res", "post", "comb")}
        loop.run_step(st)
        torch.cuda.synchronize()
        assert M.mhc_get_device_status(loop.workspace) == M.OK
        if st.pending is not None and st.pending.kind == "moe":
            xs = O.moe_finalize(f64(st.pending.gemm2_permuted), f64(st.pending.expert_weights),
                                st.pending.e2p.cpu().numpy(), f64(st.pending.shared_output))
            assert_bf16_close(f64(loop.res[b]), O.post_mix(inp["res"], xs, inp["post"], inp["comb"]), f"{st.kind} streams")
    hidden, streams = loop.hidden_out.clone(), loop.streams().clone()
    loop.run()
    torch.cuda.synchronize()
    assert torch.equal(loop.hidden_out, hidden) and torch.equal(loop.streams(), streams)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loop.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        loop.run()
    loop.hidden_out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loop.hidden_out, hidden) and torch.equal(loop.streams(), streams)
