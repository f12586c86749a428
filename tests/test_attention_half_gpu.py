"""The attention half of a quantized layer, run as a layer runs it: q/k/v
projection (W4A4 GEMM), rotation in place on slices of its output, append to
the 8-bit cache, attention, per-token INT4 codes of the heads' output, output
projection. Every stage is checked against the oracle on the GPU's own inputs
to it, eagerly and from a captured graph replayed on new activations."""
import numpy as np
import pytest
import torch

import oracle as O
import oracle.attention_oracle as AO
import rotation_post_quantization_b200 as rq
import workloads as W
from kv_util import DEV, Batch, attend

pytestmark = pytest.mark.gpu

H, G, d, P = 2, 4, 128, 16
D = H * G * d
WIDE = (G + 2) * H * d


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [40, 7, 130]), ([60, 1, 75], [60, 33, 200])])
def test_attention_half(q_lens, kv_lens):
    bt = Batch(q_lens, kv_lens, H, d, P, seed=3).to_gpu()
    N = bt.N
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    qw, ow = W.int4_packed_random(WIDE, D, 0, W.TID_WEIGHTS), W.int4_packed_random(D, D, 1, W.TID_WEIGHTS)
    sw, so = W.weight_scales(WIDE, D, 0), W.weight_scales(D, D, 1)
    dqw, dow, dsw, dso = (torch.from_numpy(x).to(DEV) for x in (qw, ow, sw, so))
    freq_h = (10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)
    freq = torch.from_numpy(freq_h).to(DEV)
    pos_h = np.concatenate([np.arange(n - m, n) for m, n in zip(q_lens, kv_lens)]).astype(np.int32)
    pos = torch.from_numpy(pos_h).to(DEV)
    qa = torch.empty(N, D // 2, dtype=torch.uint8, device=DEV)
    sa = torch.empty(N, device=DEV)
    qkv = torch.empty(N, WIDE, dtype=torch.bfloat16, device=DEV)
    raw = torch.empty_like(qkv)
    heads = qkv.view(N, (G + 2) * H, d)
    qh, kh, vh = heads[:, :G * H], heads[:, G * H:G * H + H], heads[:, G * H + H:]
    at = torch.empty(N, G * H, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(N, G * H, device=DEV)
    codes = torch.empty(N, D // 2, dtype=torch.uint8, device=DEV)
    sc = torch.empty(N, device=DEV)
    y = torch.empty(N, D, dtype=torch.bfloat16, device=DEV)
    plan = rq.Plan(D, 0)
    ws = torch.empty(rq.respin_kv_attention_workspace(bt.cache, G * H, N, max(q_lens)), dtype=torch.uint8, device=DEV)

    def layer():
        rq.w4a4_gemm(qa, sa, dqw, dsw, qkv)
        raw.copy_(qkv)
        rq.respin_qk_norm_rope(qh, kh, pos, freq, qh, kh)
        rq.respin_kv_append(bt.cache, kh, vh, bt.t_len, bt.t_table, cu=bt.t_cu)
        rq.respin_kv_attention(bt.cache, qh, bt.t_len, bt.t_table, at, ws, cu=bt.t_cu, max_q=max(q_lens), lse=lse)
        rq.respin_boundary_forward(plan, at.view(N, D), None, None, codes, sc)
        rq.w4a4_gemm(codes, sc, dow, dso, y)

    def check():
        torch.cuda.synchronize()
        assert rq.respin_device_status() == 0
        want = O.w4a4_epilogue_bits(O.w4a4_acc_fp64(qa.cpu().numpy(), qw), sa.cpu().numpy(), sw)
        assert np.array_equal(bits(raw), want)
        x = raw.view(N, -1, d).double().cpu().numpy()
        for got, part in ((qh, x[:, :G * H]), (kh, x[:, G * H:G * H + H])):
            ref, amp = AO.norm_rope(part, None, 0.0, pos_h, freq_h, False)
            # bf16, and fp32 sine and cosine
            assert (np.abs(got.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * amp).all()
        for c, s, part, tc, ts in ((bt.kc, bt.ks, kh, bt.cache.k, bt.cache.k_scale), (bt.vc, bt.vs, vh, bt.cache.v, bt.cache.v_scale)):
            AO.append(c, s, part.double().cpu().numpy(), bt.cu, bt.kv_len, bt.table, P)
            assert np.array_equal(tc.cpu().numpy(), c) and np.array_equal(ts.cpu().numpy(), s)
        out, l = attend(bt, G * H, q=qh.double().cpu().numpy())   # against the oracle, and the same bits
        assert torch.equal(out, at) and torch.equal(l, lse)
        cd, scale = O.quantize_per_token(O.bf16_bits_to_f32(bits(at.view(N, D))), 7)
        assert np.array_equal(codes.cpu().numpy(), O.pack_int4(cd))
        assert np.array_equal(sc.cpu().numpy().view(np.uint32), scale.view(np.uint32))
        assert np.array_equal(bits(y), O.w4a4_epilogue_bits(O.w4a4_acc_fp64(codes.cpu().numpy(), ow), scale, so))

    def fill(seed):
        g.manual_seed(seed)
        qa.copy_(torch.randint(0, 256, qa.shape, generator=g, device=DEV, dtype=torch.uint8))
        sa.copy_(torch.rand(N, generator=g, device=DEV) + 0.5)

    fill(1)
    layer()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    fill(2)
    graph.replay()
    check()
    plan.destroy()
