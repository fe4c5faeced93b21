"""The 4-bit weight operators against plain fp64 forms: matrix-vector products and the
MoE layer for a few tokens."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from mixture_experts_layer_align_gb300 import inputs

pytestmark = pytest.mark.gpu


def tensor(moe, parts, group):
    codes, scales, zeros = parts
    return moe.W4Tensor(codes.cuda(), scales.cuda(), None if zeros is None else zeros.cuda(),
                        group=group)


def draw_x(T, K, seed=0):
    g = torch.Generator().manual_seed(seed + 101)
    return torch.randn(T, K, generator=g).to(torch.bfloat16)


def check_matvec(got, x, v, out_dtype):
    want, mag = ref.matvec(x, v)
    err = np.abs(got.float().cpu().numpy() - want)
    bound = ref.sum_bound(x.shape[1]) * mag + 1e-30
    if out_dtype == torch.bfloat16:
        bound += ref.BF16 * (np.abs(want) + bound)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.2f} of the bound"


MATVEC = [
    # T, K, N, group, scale, zeros, out
    (1, 32, 1, 32, "fp32", False, "bf16"),
    (1, 32, 7, 128, "bf16", True, "fp32"),       # one short group
    (2, 96, 16, 64, "fp32", True, "bf16"),       # a short last group
    (3, 160, 33, 128, "bf16", False, "fp32"),
    (5, 1056, 1027, 128, "fp32", True, "fp32"),
    (7, 2048, 129, 32, "bf16", True, "bf16"),
    (8, 4096, 64, 128, "fp32", False, "fp32"),
    (9, 4128, 31, 64, "bf16", False, "bf16"),
    (16, 736, 300, 32, "fp32", True, "fp32"),
    (17, 7200, 130, 128, "bf16", True, "fp32"),
    (24, 512, 2049, 64, "fp32", False, "bf16"),
    (33, 1888, 65, 32, "bf16", False, "fp32"),
    (40, 14336, 48, 128, "fp32", True, "fp32"),
    (64, 2080, 257, 64, "bf16", True, "fp32"),
    (65, 64, 5, 32, "fp32", False, "fp32"),
    (200, 416, 100, 128, "bf16", True, "bf16"),
    (1, 28672, 40, 128, "bf16", False, "fp32"),
    (1, 4096, 20000, 128, "bf16", True, "fp32"),
    (4, 32, 9001, 32, "bf16", True, "bf16"),
]


@pytest.mark.parametrize("T,K,N,group,scale,zeros,out", MATVEC)
def test_matvec(gpu_lib, T, K, N, group, scale, zeros, out):
    parts = ref.make_w4((N, K), group, scale, zeros, seed=T + N)
    x = draw_x(T, K, seed=K)
    dt = torch.float32 if out == "fp32" else torch.bfloat16
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, group), out_dtype=dt)
    assert got.shape == (T, N) and got.dtype == dt
    check_matvec(got, x, ref.values(*parts, group), dt)


def test_matvec_random_shapes(gpu_lib):
    rng = np.random.default_rng(71)
    for i in range(40):
        T = int(np.exp(rng.uniform(0, np.log(80))))
        K = 32 * int(np.exp(rng.uniform(0, np.log(150))))
        N = int(np.exp(rng.uniform(0, np.log(900))))
        group = int(rng.choice([32, 64, 128]))
        test_matvec(gpu_lib, T, K, N, group, str(rng.choice(["fp32", "bf16"])),
                    bool(rng.integers(2)), str(rng.choice(["fp32", "bf16"])))


def test_every_code_and_zero_point_is_exact(gpu_lib):
    """x picks one column at a time: the product is the weight's value itself."""
    K, group = 64, 32
    codes = torch.arange(256, dtype=torch.uint8).repeat_interleave(16)[:, None].expand(-1, K // 2)
    zeros = torch.arange(16, dtype=torch.uint8).repeat(256)[:, None].expand(-1, 2)
    scales = torch.full((4096, 2), 1.0)
    scales[:, 1] = -3.0
    parts = codes.contiguous(), scales, zeros.contiguous()
    x = torch.zeros(4, K, dtype=torch.bfloat16)
    cols = (0, 31, 32, 63)
    for t, k in enumerate(cols):
        x[t, k] = 1.0
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, group), out_dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy(), ref.values(*parts, group)[:, list(cols)].T)


def test_each_column_is_read_once(gpu_lib):
    """One-hot tokens walk over every column of a short-grouped row."""
    K, N, group = 416, 24, 128
    parts = ref.make_w4((N, K), group, "fp32", True, seed=3)
    x = torch.eye(K, dtype=torch.bfloat16)
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, group), out_dtype=torch.float32)
    want = ref.values(*parts, group).astype(np.float32).T
    assert np.allclose(got.cpu().numpy(), want, rtol=2.0 ** -22, atol=0)


def test_matvec_non_finite_values_stay_in_their_row_and_column(gpu_lib):
    T, K, N, group = 13, 256, 50, 64
    codes, scales, zeros = ref.make_w4((N, K), group, "fp32", True, seed=4)
    x = draw_x(T, K)
    v = ref.values(codes, scales, zeros, group)
    x[3, 17], x[9, 200] = float("nan"), float("inf")
    scales[21, 2], scales[44, 0] = float("nan"), float("inf")
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, (codes, scales, zeros), group),
                                out_dtype=torch.float32).cpu().numpy()
    assert np.isnan(got[3]).all() and np.isnan(got[:, 21]).all()
    assert not np.isfinite(got[:, 44]).any()
    code = np.stack([codes.numpy() & 15, codes.numpy() >> 4], -1).reshape(N, K)[:, 200]
    sign = np.sign(code.astype(int) - zeros.numpy()[:, 200 // group])
    plain = np.setdiff1d(np.arange(N), [21, 44])
    # inf x weight: infinite of the weight's sign, NaN where the weight is zero
    want = np.where(sign == 0, np.nan, sign * np.inf)[plain]
    assert np.array_equal(got[9, plain], want, equal_nan=True)
    rows = np.setdiff1d(np.arange(T), [3, 9])
    check_matvec(torch.from_numpy(got[np.ix_(rows, plain)]), x[rows], v[plain], torch.float32)


def test_matvec_zero_tokens_and_zero_weights(gpu_lib):
    parts = ref.make_w4((9, 64), 32, "fp32", False, seed=5)
    w = tensor(gpu_lib, parts, 32)
    assert gpu_lib.moe_w4_matvec(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                                 w).shape == (0, 9)
    codes = torch.full((9, 32), 0x88, dtype=torch.uint8)
    y = gpu_lib.moe_w4_matvec(draw_x(3, 64).cuda(), tensor(gpu_lib, (codes, parts[1], None), 32))
    assert not y.any()


def test_matvec_writes_its_own_output_only(gpu_lib):
    """Rows of an output in the middle of a larger buffer; the rest keeps its contents."""
    T, K, N = 11, 160, 37
    parts = ref.make_w4((N, K), 64, "bf16", True, seed=6)
    x = draw_x(T, K)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((T + 2, N), 7.0, dtype=dt, device="cuda")
        gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, 64), out=buf[1:-1])
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        check_matvec(buf[1:-1], x, ref.values(*parts, 64), dt)


def test_matvec_is_the_same_every_time_and_on_a_side_stream(gpu_lib):
    parts = ref.make_w4((1000, 4096), 128, "bf16", True, seed=7)
    w = tensor(gpu_lib, parts, 128)
    x = draw_x(6, 4096).cuda()
    first = gpu_lib.moe_w4_matvec(x, w, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [gpu_lib.moe_w4_matvec(x, w, out_dtype=torch.float32, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(first, a) for a in again)


# ---------------------------------------------------------------- the layer

LAYER = [
    # T, H, I, E, k, group, scale, zeros, routing, renorm
    (1, 32, 32, 1, 1, 32, "fp32", False, "uniform", True),
    (1, 128, 64, 4, 4, 128, "bf16", True, "uniform", False),
    (3, 416, 224, 5, 3, 32, "fp32", True, "uniform", False),
    (4, 128, 256, 8, 2, 128, "fp32", False, "uniform", True),
    (7, 96, 160, 3, 1, 64, "bf16", True, "uniform", True),
    (8, 256, 96, 16, 8, 64, "fp32", True, "zipf", True),
    (9, 544, 416, 6, 2, 128, "bf16", False, "zipf", True),
    (16, 320, 128, 40, 5, 32, "bf16", True, "uniform", False),
    (17, 160, 288, 2, 2, 128, "fp32", True, "uniform", True),
    (33, 288, 352, 4, 1, 64, "fp32", False, "zipf", True),    # > 8 tokens per expert
    (64, 256, 192, 8, 2, 32, "bf16", True, "uniform", True),
    (64, 1056, 96, 300, 6, 128, "fp32", False, "uniform", True),  # E > 256
    (65, 64, 32, 1, 1, 32, "fp32", True, "uniform", True),    # all on one expert
    (300, 128, 64, 7, 3, 64, "bf16", True, "zipf", True),
    (2, 2048, 768, 16, 8, 128, "bf16", False, "uniform", True),
    (1, 96, 64, 1024, 40, 32, "fp32", True, "uniform", True),  # k > 32, the most experts
]


def run_layer(moe, T, H, I, E, k, group, scale, zeros, routing, renorm, seed=0, **kw):
    p13 = ref.make_w4((E, 2 * I, H), group, scale, zeros, seed=seed + 1)
    p2 = ref.make_w4((E, H, I), group, scale, zeros, seed=seed + 2)
    a = inputs.make_activations(T, H, E, routing, seed=seed)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    wts = torch.empty(T, k, dtype=torch.float32, device="cuda")
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    args = (a.x.cuda(), a.logits.cuda(), tensor(moe, p13, group), tensor(moe, p2, group), k, renorm)
    out = moe.moe_w4_forward(*args, topk_ids_out=ids, topk_w_out=wts, counts_out=counts, **kw)
    return a, p13, p2, args, out, ids, wts, counts


def check_layer(a, p13, p2, k, renorm, group, out, ids=None, wts=None, counts=None):
    want = ref.layer(a.x, a.logits, ref.values(*p13, group), ref.values(*p2, group), k, renorm)
    H, I = a.x.shape[1], p2[0].shape[2] * 2
    if ids is not None:
        assert np.array_equal(ids.cpu().numpy(), want["ids"])
        assert np.array_equal(counts.cpu().numpy(), want["counts"])
        assert np.allclose(wts.cpu().numpy(), want["weights"], rtol=1e-5, atol=1e-7)
    err = np.abs(out.float().cpu().numpy() - want["out"])
    # h rounded to bf16 (the SiLU product at most doubles the sums' relative error and is
    # dominated by that rounding), the sums of the second product, the result rounded
    bound = (2 * ref.BF16 + ref.sum_bound(H) + ref.sum_bound(I)) * want["mag"] \
        + ref.BF16 * np.abs(want["out"]) + 1e-30
    assert np.all(err <= bound), f"worst {np.max(err / bound):.2f} of the bound"
    # the two roundings to bf16 are independent and of rms at most 2^-8 / sqrt(3) each
    if err.size >= 256:
        norm = np.linalg.norm(err) / np.linalg.norm(want["out"])
        assert norm <= ref.BF16, f"error {norm:.2e} of the norm"


@pytest.mark.parametrize("T,H,I,E,k,group,scale,zeros,routing,renorm", LAYER)
def test_layer(gpu_lib, T, H, I, E, k, group, scale, zeros, routing, renorm):
    a, p13, p2, _, out, ids, wts, counts = run_layer(gpu_lib, T, H, I, E, k, group, scale, zeros,
                                                     routing, renorm, seed=T)
    assert out.shape == (T, H) and out.dtype == torch.bfloat16
    check_layer(a, p13, p2, k, renorm, group, out, ids, wts, counts)


def test_layer_random_shapes(gpu_lib):
    rng = np.random.default_rng(72)
    for i in range(30):
        T = int(np.exp(rng.uniform(0, np.log(80))))
        E = int(np.exp(rng.uniform(0, np.log(64))))
        k = int(rng.integers(1, min(E, 8) + 1))
        H, I = (32 * int(np.exp(rng.uniform(0, np.log(24)))) for _ in range(2))
        test_layer(gpu_lib, T, H, I, E, k, int(rng.choice([32, 64, 128])),
                   str(rng.choice(["fp32", "bf16"])), bool(rng.integers(2)),
                   str(rng.choice(["uniform", "zipf"])), bool(rng.integers(2)))


def test_layer_equals_its_steps(gpu_lib):
    """E = 1, k = 1 is the matvec chain w2 (SiLU(gate) up)."""
    T, H, I, group = 5, 512, 384, 64
    p13, p2 = (ref.make_w4((1, n, k), group, "fp32", True, seed=s)
               for n, k, s in ((2 * I, H, 1), (H, I, 2)))
    a = inputs.make_activations(T, H, 1, "uniform", seed=9)
    x = a.x.cuda()
    w13, w2 = tensor(gpu_lib, p13, group), tensor(gpu_lib, p2, group)
    out = gpu_lib.moe_w4_forward(x, a.logits.cuda(), w13, w2, 1)
    flat = [tensor(gpu_lib, [t if t is None else t[0] for t in p], group) for p in (p13, p2)]
    gu = gpu_lib.moe_w4_matvec(x, flat[0], out_dtype=torch.float32)
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    y = gpu_lib.moe_w4_matvec(h.to(torch.bfloat16), flat[1], out_dtype=torch.float32)
    assert torch.allclose(out.float(), y, rtol=2 * ref.BF16,
                          atol=2 * ref.BF16 * y.abs().max().item())


def test_layer_workspace_reuse_and_determinism(gpu_lib):
    """A dirty workspace, and calls of other sizes in it, leave no trace."""
    moe = gpu_lib
    big = moe.alloc_w4_workspace(64, 1024, 512, 64, 8)
    big.fill_(0xAB)
    case = (23, 256, 192, 12, 4, 64, "bf16", True, "zipf", True)
    a, p13, p2, args, first, *_ = run_layer(moe, *case, seed=5, workspace=big)
    run_layer(moe, 40, 128, 320, 30, 3, 32, "fp32", False, "uniform", True, seed=6, workspace=big)
    again = moe.moe_w4_forward(*args, workspace=big)
    assert torch.equal(first, again)
    assert moe.moe_check_status(big) == 0
    check_layer(a, p13, p2, 4, True, 64, again)


def test_layer_non_finite_tokens_stay_alone(gpu_lib):
    T, H, I, E, k, group = 20, 128, 96, 4, 2, 32
    p13, p2 = ref.make_w4((E, 2 * I, H), group, seed=1), ref.make_w4((E, H, I), group, seed=2)
    a = inputs.make_activations(T, H, E, "uniform", seed=8)
    args = (a.logits.cuda(), tensor(gpu_lib, p13, group), tensor(gpu_lib, p2, group), k)
    good = gpu_lib.moe_w4_forward(a.x.cuda(), *args)
    x = a.x.clone()
    x[2, 5] = float("nan")
    x[11] = float("inf")
    got = gpu_lib.moe_w4_forward(x.cuda(), *args)
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[11]).any()
    rest = [t for t in range(T) if t not in (2, 11)]
    assert torch.equal(got[rest], good[rest])


def test_layer_graph_replay_and_side_stream(gpu_lib):
    moe = gpu_lib
    a, p13, p2, args, first, *_ = run_layer(moe, 6, 256, 128, 16, 4, 64, "bf16", True, "uniform",
                                            True, seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.moe_w4_forward(*args, stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    ws = moe.alloc_w4_workspace(6, 256, 128, 16, 4)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_w4_forward(*args, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_layer_zero_tokens(gpu_lib):
    p13, p2 = ref.make_w4((2, 64, 32), 32, seed=1), ref.make_w4((2, 32, 32), 32, seed=2)
    out = gpu_lib.moe_w4_forward(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"),
                                 torch.empty(0, 2, device="cuda"), tensor(gpu_lib, p13, 32),
                                 tensor(gpu_lib, p2, 32), 1)
    assert out.shape == (0, 32)


def test_binding_refusals(gpu_lib):
    moe = gpu_lib
    codes, scales, zeros = (t.cuda() for t in ref.make_w4((8, 64), 32, "fp32", True, seed=1))
    w = moe.W4Tensor(codes, scales, zeros, group=32)
    x = draw_x(2, 64).cuda()
    for bad in (lambda: moe.W4Tensor(codes, scales, zeros, group=48),
                lambda: moe.W4Tensor(codes, scales, zeros, group=64),          # scales' shape
                lambda: moe.W4Tensor(codes.cpu(), scales, zeros, group=32),
                lambda: moe.W4Tensor(codes, scales.half(), zeros, group=32),
                lambda: moe.W4Tensor(codes, scales, zeros.int(), group=32),
                lambda: moe.W4Tensor(codes.t(), scales, zeros, group=32),
                lambda: moe.moe_w4_matvec(x.float(), w),
                lambda: moe.moe_w4_matvec(x[:, :32].contiguous(), w),
                lambda: moe.moe_w4_matvec(x, w, out=torch.empty(2, 7, device="cuda")),
                lambda: moe.moe_w4_matvec(x, w, out_dtype=torch.float16),
                lambda: moe.moe_w4_matvec(x, w, out=torch.empty(2, 8, device="cuda"),
                                          out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            bad()
    odd = ref.make_w4((8, 48), 32, "fp32", False, seed=2)  # K % 32 != 0
    with pytest.raises(moe.MoeError):
        moe.moe_w4_matvec(draw_x(2, 48).cuda(), tensor(moe, odd, 32))
