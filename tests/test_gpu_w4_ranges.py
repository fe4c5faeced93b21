"""The 4-bit weight operators where their paths change: token counts around the block
sizes, more jobs than thread blocks, K split over clusters, values of every magnitude."""
import numpy as np
import pytest
import torch

import w4_ref as ref
from mixture_experts_layer_align_gb300 import inputs
from test_gpu_w4 import check_layer, check_matvec, draw_x, run_layer, tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("group", [32, 128])
def test_matvec_token_counts(gpu_lib, T, group):
    K, N = 1312, 200
    parts = ref.make_w4((N, K), group, "bf16", True, seed=T)
    x = draw_x(T, K, seed=T)
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, group), out_dtype=torch.float32)
    check_matvec(got, x, ref.values(*parts, group), torch.float32)


@pytest.mark.parametrize("T,K,N,group,zeros", [
    (1, 64, 90000, 32, True),      # one token, every thread block takes several tiles
    (1, 544, 80001, 128, False),
    (8, 64, 90000, 64, True),
    (16, 96, 70001, 32, False),
    (40, 288, 30001, 64, True),    # two token blocks, shared rows
    (200, 416, 9001, 128, True),
])
def test_matvec_more_tiles_than_thread_blocks(gpu_lib, T, K, N, group, zeros):
    parts = ref.make_w4((N, K), group, "fp32", zeros, seed=11)
    x = draw_x(T, K, seed=12)
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, group), out_dtype=torch.float32)
    check_matvec(got, x, ref.values(*parts, group), torch.float32)


@pytest.mark.parametrize("T", [1, 5, 16, 40])
@pytest.mark.parametrize("K", [256, 512, 1024, 2048, 4096, 4128, 8160, 14368])
def test_matvec_k_split(gpu_lib, T, K):
    """Few rows: K goes over clusters of up to 16 blocks, whose slices need not be equal."""
    parts = ref.make_w4((130, K), 64, "fp32", True, seed=K)
    x = draw_x(T, K, seed=13)
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, parts, 64), out_dtype=torch.float32)
    check_matvec(got, x, ref.values(*parts, 64), torch.float32)


@pytest.mark.parametrize("T", [1, 6, 20])
@pytest.mark.parametrize("low,high", [(-110, -90), (90, 110), (-20, 20), (-133, -120)])
def test_matvec_magnitudes(gpu_lib, T, low, high):
    """x over a range of powers of two.  Of the largest |x| of 256 columns the pieces drop
    less than 2^-31, so a column is off by that much times its weight at most."""
    K, N, group = 800, 70, 32
    codes, scales, zeros = ref.make_w4((N, K), group, "fp32", True, seed=21)
    g = torch.Generator().manual_seed(22)
    power = torch.randint(low, high + 1, (T, K), generator=g).double()
    x = (torch.randn(T, K, generator=g).double() * 2.0 ** power).to(torch.bfloat16)
    v = ref.values(codes, scales, zeros, group)
    got = gpu_lib.moe_w4_matvec(x.cuda(), tensor(gpu_lib, (codes, scales, zeros), group),
                                out_dtype=torch.float32)
    want, mag = ref.matvec(x, v)
    # codes, not their distances from the zero point, multiply what is dropped
    spread = 15 * np.repeat(scales.double().numpy(), group, axis=1)[:, :K]
    top = np.abs(x.double().numpy())
    dropped = np.zeros_like(want)
    # MMAs and sums work on codes and x, so their rounding is relative to that too
    worst = top @ spread.T
    for k in range(0, K, 256):
        dropped += 2.0 ** -31 * np.outer(top[:, k:k + 256].max(1), spread[:, k:k + 256].sum(1))
    bound = 2 * dropped + ref.sum_bound(K) * worst + 2.0 ** -140
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.2f} of the bound"


def test_matvec_one_token_equals_its_row_of_many(gpu_lib):
    """A token alone is split by the kernel that uses it: the same sums, to their rounding."""
    K, N = 4096, 300
    parts = ref.make_w4((N, K), 128, "bf16", True, seed=31)
    w = tensor(gpu_lib, parts, 128)
    x = draw_x(6, K, seed=32)
    v = ref.values(*parts, 128)
    for t in range(6):
        y = gpu_lib.moe_w4_matvec(x[t:t + 1].cuda(), w, out_dtype=torch.float32)
        check_matvec(y, x[t:t + 1], v, torch.float32)


def test_matvec_non_finite_single_token(gpu_lib):
    K, N = 640, 40
    parts = ref.make_w4((N, K), 128, "fp32", True, seed=33)
    w = tensor(gpu_lib, parts, 128)
    x = draw_x(1, K)
    x[0, 300] = float("nan")
    assert gpu_lib.moe_w4_matvec(x.cuda(), w).isnan().all()
    x[0, 300] = float("inf")
    y = gpu_lib.moe_w4_matvec(x.cuda(), w).float().cpu().numpy()
    sign = np.sign(ref.values(*parts, 128)[:, 300])
    assert np.array_equal(y[0], np.where(sign == 0, np.nan, sign * np.inf), equal_nan=True)


def test_matvec_strided_x_is_refused(gpu_lib):
    parts = ref.make_w4((16, 64), 32, seed=1)
    w = tensor(gpu_lib, parts, 32)
    wide = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gpu_lib.moe_w4_matvec(wide[:, :64], w)
    with pytest.raises(ValueError):
        gpu_lib.moe_w4_matvec(wide[:, ::2], w)


LAYER = [
    # T, H, I, E, k, routing: pairs around the joint front kernel's limit, block sizes by the
    # pairs of an expert, more jobs than thread blocks
    (256, 64, 32, 16, 1, "uniform"),
    (257, 64, 32, 16, 1, "uniform"),
    (32, 96, 64, 256, 8, "zipf"),
    (32, 96, 64, 257, 8, "uniform"),
    (48, 128, 64, 8, 1, "uniform"),    # 6 pairs an expert
    (49, 128, 64, 8, 1, "uniform"),
    (96, 128, 64, 8, 1, "zipf"),       # 12
    (97, 128, 64, 8, 1, "uniform"),
    (64, 256, 512, 64, 4, "uniform"),
    (40, 1024, 96, 4, 3, "zipf"),
    (1, 4096, 64, 2, 2, "uniform"),    # K split over clusters
    (1, 64, 4128, 3, 2, "uniform"),
]


@pytest.mark.parametrize("T,H,I,E,k,routing", LAYER)
def test_layer_paths(gpu_lib, T, H, I, E, k, routing):
    a, p13, p2, _, out, ids, wts, counts = run_layer(gpu_lib, T, H, I, E, k, 32, "fp32", True,
                                                     routing, True, seed=T + E)
    check_layer(a, p13, p2, k, True, 32, out, ids, wts, counts)


def test_layer_large_h(gpu_lib):
    """h beyond the range of fp16."""
    T, H, I, E, k = 6, 256, 160, 4, 2
    p13 = ref.make_w4((E, 2 * I, H), 64, "fp32", False, seed=41)
    p2 = ref.make_w4((E, H, I), 64, "fp32", False, seed=42)
    a = inputs.make_activations(T, H, E, "uniform", seed=43)
    a.x *= 4096
    out = gpu_lib.moe_w4_forward(a.x.cuda(), a.logits.cuda(), tensor(gpu_lib, p13, 64),
                                 tensor(gpu_lib, p2, 64), k)
    want = ref.layer(a.x, a.logits, ref.values(*p13, 64), ref.values(*p2, 64), k, True)
    assert np.abs(want["out"]).max() > 65504
    check_layer(a, p13, p2, k, True, 64, out)


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (40, 64, 8)])
def test_layer_ties_go_to_the_lower_expert(gpu_lib, T, E, k):
    """Equal logits, and the same from the joint front kernel and the separate ones."""
    H, I = 64, 32
    p13, p2 = ref.make_w4((E, 2 * I, H), 32, seed=1), ref.make_w4((E, H, I), 32, seed=2)
    x = draw_x(T, H)
    logits = torch.zeros(T, E)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gpu_lib.moe_w4_forward(x.cuda(), logits.cuda(), tensor(gpu_lib, p13, 32),
                           tensor(gpu_lib, p2, 32), k, topk_ids_out=ids)
    assert torch.equal(ids.cpu(), torch.arange(k, dtype=torch.int32).expand(T, k))


def test_matvec_scratch_of_its_own_on_each_stream(gpu_lib):
    """Calls with one weight on two streams at a time, and in a graph replayed beside calls
    of another size, do not disturb one another."""
    K, N = 4096, 3000
    parts = ref.make_w4((N, K), 128, "bf16", True, seed=51)
    w = tensor(gpu_lib, parts, 128)
    xs = [draw_x(T, K, seed=T).cuda() for T in (12, 40)]
    want = [gpu_lib.moe_w4_matvec(x, w) for x in xs]
    graph, y = torch.cuda.CUDAGraph(), torch.empty_like(want[0])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(20):
            gpu_lib.moe_w4_matvec(xs[0], w, out=y)
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(gpu_lib.moe_w4_matvec(xs[i], w))
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
    assert torch.equal(y, want[0])
