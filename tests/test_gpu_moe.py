"""The mixture-of-experts layer (q8_moe) against the binary64 definition: the
experts chosen, their weights, and the outputs within what fp32 sums may be
off (decode_ref.moe)."""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu


def experts(E, H, F, seed):
    r = np.random.default_rng(seed)
    out = []
    for rows, K in ((2 * F, H), (H, F)):
        c = r.integers(-127, 128, (E, rows, K), dtype=np.int8)
        s = (r.uniform(0.3, 1.0, (E, rows, K // 32)) * 0.03 / 64).astype(np.float16)
        out += [c, s]
    return out


def run(T, E, H, F, k, renorm=True, seed=0, x=None, logits=None, status=0, stream=None, xs=1.0):
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(seed + 100)
    c13, s13, c2, s2 = experts(E, H, F, seed)
    if x is None:
        x = torch.from_numpy((r.standard_normal((T, H)) * xs).astype(np.float32)).to(torch.bfloat16).cuda()
    if logits is None:
        logits = r.standard_normal((T, E)).astype(np.float32) * 2
    lg = torch.from_numpy(logits).cuda() if isinstance(logits, np.ndarray) else logits
    dev = [torch.from_numpy(a).cuda() for a in (c13, s13, c2, s2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    y, ids, w = q8.q8_moe(x, lg, *dev, k, renorm=renorm, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    v13, v2 = ref.values(c13, s13.view(np.uint16)), ref.values(c2, s2.view(np.uint16))
    want, tol, wi, ww = ref.moe(x.double().cpu().numpy(), lg.cpu().numpy(), v13, v2, k, renorm)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert np.all(np.abs(w.double().cpu().numpy() - ww) <= 2.0 ** -20 * ww)
    got = y.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.all(err <= tol), (err.max(), tol[err > tol].min())
    if np.any(want):
        # typical errors are far below the bound: binary32 outputs keep their digits
        assert np.linalg.norm(got - want) <= 2.0 ** -19 * np.linalg.norm(want)
    return y, ids, w, dev, x, lg


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32])
def test_tokens(T):
    run(T, 8, 256, 96, 3, seed=T)


@pytest.mark.parametrize("H,F", [(32, 32), (64, 1376), (288, 32), (544, 160), (1024, 512), (4096, 64)])
def test_widths(H, F):
    # rows of scales that start on odd 2-byte offsets, partial chunks of 256, partial tiles of 64 rows
    run(5, 4, H, F, 2, seed=H + F)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (16, 16), (33, 1), (130, 8), (512, 4)])
@pytest.mark.parametrize("renorm", [True, False])
def test_experts(E, k, renorm):
    run(6, E, 64, 64, k, renorm=renorm, seed=E + k)


def test_every_token_on_every_expert():
    run(32, 2, 512, 256, 2, seed=1)
    run(31, 4, 96, 352, 4, renorm=False, seed=2)


def test_ties_go_to_the_lower_index():
    lg = np.zeros((3, 40), dtype=np.float32)
    lg[1, 35] = 1.0
    lg[2, ::2] = -0.0
    y, ids, *_ = run(3, 40, 64, 32, 3, logits=lg)
    assert ids.cpu().tolist() == [[0, 1, 2], [35, 0, 1], [0, 1, 2]]


def test_masked_experts_and_empty_tokens():
    from block_quantized_int8_gb300 import q8
    lg = np.random.default_rng(3).standard_normal((5, 20)).astype(np.float32)
    lg[0] = -np.inf                       # no expert at all
    lg[1, 2:] = -np.inf                   # fewer than top_k
    lg[2] = np.finfo(np.float32).min      # all at the type's lowest value: like any tie
    lg[3, 7] = np.inf
    y, ids, w, *_ = run(5, 20, 64, 64, 4, logits=lg)
    assert not y[0].any() and ids[0].tolist() == [-1] * 4
    assert ids[1, 2:].tolist() == [-1, -1] and ids[2].tolist() == [0, 1, 2, 3]
    run(5, 20, 64, 64, 4, logits=lg, renorm=False)
    lg[4, 3] = np.nan
    run(5, 20, 64, 64, 4, logits=lg, status=q8.Q8_DEV_NONFINITE)
    run(2, 20, 64, 64, 4, logits=np.full((2, 20), -np.inf, dtype=np.float32))


@pytest.mark.parametrize("xs", [1e-12, 1e-3, 300.0])
def test_activation_ranges(xs):
    run(4, 4, 128, 128, 2, seed=5, xs=xs)


def test_strides_and_another_stream():
    r = np.random.default_rng(8)
    wide = torch.from_numpy(r.standard_normal((6, 400)).astype(np.float32)).to(torch.bfloat16).cuda()
    lg = torch.from_numpy(r.standard_normal((6, 50)).astype(np.float32)).cuda()
    run(6, 12, 96, 64, 3, x=wide[:, 8:104], logits=lg[:, 5:17], stream=torch.cuda.Stream())


def test_repeats_and_graph_replays_with_other_logits():
    from block_quantized_int8_gb300 import q8
    y, ids, w, dev, x, lg = run(20, 24, 512, 512, 4, seed=9)
    ws = q8.workspace(q8.q8_moe_workspace_size(20, 24, 512, 512, 4))
    out = torch.empty_like(y)
    for _ in range(20):
        q8.q8_moe(x, lg, *dev, 4, y=out, ws=ws)
        assert torch.equal(out, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q8.q8_moe(x, lg, *dev, 4, y=out, ws=ws)
    for seed in range(3):
        lg.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((20, 24)).astype(np.float32)))
        g.replay()
        want, _, _ = q8.q8_moe(x, lg, *dev, 4)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_router_by_the_skinny_matmul(oracle):
    # the router's logits as q8_gemm_skinny leaves them
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(10)
    rq, rs, _ = oracle.quantize_rows((r.standard_normal((16, 256)) * 0.1).astype(np.float32))
    x = torch.from_numpy(r.standard_normal((3, 256)).astype(np.float32)).to(torch.bfloat16).cuda()
    lg = q8.q8_gemm_skinny(torch.from_numpy(rq).cuda(), torch.from_numpy(rs.view(np.int16)).cuda(), x)
    run(3, 16, 256, 96, 2, x=x, logits=lg)
