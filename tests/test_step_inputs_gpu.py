"""8-bit activation checkpoints, weight gradients and attention on the GPU, against plain
float64 forms."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import step_inputs_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def B(lib):
    from matrix_orthogonalising_optimizer_03_b200 import binding
    return binding


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from matrix_orthogonalising_optimizer_03_b200 import binding
    return binding.load()


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets_of(lengths, first=0):
    off = [first]
    for n in lengths:
        off.append(off[-1] + n)
    return off


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("rows,cols,ld,dtype", [
    (1, 1, 1, F32), (1, 1, 1, BF16), (3, 31, 31, BF16), (5, 32, 32, F32), (7, 33, 40, BF16),
    (2, 9001, 9001, BF16), (3, 20000, 20008, F32), (1000, 8, 8, BF16), (64, 255, 255, F32), (129, 1021, 1024, BF16), (33, 2048, 2053, F32), (300, 320, 320, BF16)])
def test_store_and_restore_follow_the_definition(B, rows, cols, ld, dtype):
    g = gen_of(rows * 1000 + cols)
    x = torch.zeros(rows, ld, device="cuda", dtype=dtype)[:, :cols]
    x.copy_(randn(g, rows, cols) * torch.exp(3 * randn(g, 1, cols)))
    x[0, 0] = 0.0
    if rows > 2:
        x[1] = 0.0                                # whole groups of zeros
        x[2, :1] = 2.0 ** -40                     # a power of two as the largest magnitude
    ck = B.new_act8(rows, cols)
    ck.q.fill_(99)
    ck.exps.fill_(98)
    B.act8_store([x], [ck])
    q, byte = ref.store(x)
    assert torch.equal(ck.q[:, :cols].cpu(), q)
    assert torch.equal(ck.exps[:, :byte.shape[1]].cpu(), byte)
    assert bool((ck.q[:, cols:] == 99).all()) and bool((ck.exps[:, byte.shape[1]:] == 98).all())
    for dt in (BF16, F32):
        wide = torch.full((rows, ld), 7.0, device="cuda", dtype=dt)
        B.act8_restore([ck], [wide[:, :cols]])
        assert torch.equal(wide[:, :cols].cpu().double(), ref.restore(q, byte))    # exact in both types
        assert bool((wide[:, cols:] == 7).all())


def test_store_extremes(B):
    """Zeros, subnormals, the largest finite values, values that round past 127, NaN and
    infinities: each group by the definition."""
    x = torch.zeros(8, 96, device="cuda")
    x[0, 3] = 1e-45
    x[1, 40] = 2.0 ** -126
    x[2, 5], x[2, 6] = 3.4028234e38, -1.0
    x[3, 1], x[3, 2], x[3, 3] = 127.9, -127.9, 0.5      # 0.5, 1.5: ties to even
    x[3, 4] = 1.5
    x[4, 33] = math.nan
    x[5, 70] = -math.inf
    x[6] = torch.arange(96, device="cuda").float() - 48
    ck = B.new_act8(8, 96)
    B.act8_store([x], [ck])
    q, byte = ref.store(x)
    assert torch.equal(ck.q.cpu()[:, :96], q) and torch.equal(ck.exps.cpu()[:, :3], byte)
    assert byte[4, 1] == 255 and byte[5, 2] == 255 and int((byte == 255).sum()) == 2
    y = torch.zeros_like(x)
    B.act8_restore([ck], [y])
    want = ref.restore(q, byte)
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want)) and torch.equal(
        y.cpu().double().nan_to_num(0), want.nan_to_num(0))
    ck.exps[7, 0] = 0                                   # byte 0 is a scale of zero
    ck.q[7, 0] = 64
    B.act8_restore([ck], [y])
    assert float(y[7, 0]) == 0


def test_store_takes_lists_in_several_launches(B):
    xs, cks = [], []
    for i in range(150):
        xs.append(randn(gen_of(i), (i * 7) % 40, 1 + (i * 13) % 70).to(BF16 if i % 2 else F32))
        cks.append(B.new_act8(*xs[-1].shape))
    ys = [torch.empty_like(x) for x in xs]
    B.act8_store(xs, cks)
    B.act8_restore(cks, ys)
    for x, y in zip(xs, ys):
        if x.numel():
            assert torch.equal(y.cpu().double(), ref.restore(*ref.store(x)))
    B.act8_store([], [])
    B.act8_restore([], [])


def test_rows_that_overlap_are_refused(B):
    """A broadcast row and overlapping windows, as source and as target; nothing is launched."""
    row = torch.ones(64, device="cuda")
    ck = B.new_act8(8, 64)
    before = ck.q.clone()
    for x in (row.expand(8, 64), torch.ones(200, device="cuda").as_strided((8, 64), (16, 1))):
        for call in (lambda: B.act8_store([x], [ck]), lambda: B.act8_restore([ck], [x])):
            with pytest.raises(B.MuonError) as e:
                call()
            assert e.value.status == 2
    torch.cuda.synchronize()
    assert torch.equal(ck.q, before) and bool((row == 1).all())
    one = torch.ones(8, 200, device="cuda").t()[:1]             # a single row, of stride 1
    B.act8_store([row[None, :8].expand(1, 8)], [B.new_act8(1, 8)])
    with pytest.raises(B.MuonError):
        B.act8_store([one], [B.new_act8(1, 8)])                 # its columns are 200 apart


# ---------------------------------------------------------------- weight gradients
def stored(B, gen, tokens, inn, scale=1.0):
    ck = B.new_act8(tokens, inn)
    x = (randn(gen, tokens, inn) * scale * torch.exp(randn(gen, 1, inn))).to(BF16)
    if tokens:
        B.act8_store([x], [ck])
    return ck, ref.restore(ck.q[:, :inn], ck.exps[:, :(inn + 31) // 32]).cuda()


def dy_of(gen, tokens, out, pad=0):
    dy = torch.zeros(tokens, (out + 7) // 8 * 8 + pad, device="cuda", dtype=BF16)[:, :out]
    dy.copy_(randn(gen, tokens, out))
    return dy


WGRAD = [
    # out, in, tokens per group
    (8, 8, [1]), (1, 1, [3]), (64, 64, [64]), (128, 256, [64]), (129, 257, [65]), (130, 40, [63]),
    (512, 320, [1000]), (100, 33, [2, 0, 129]), (320, 512, [64, 1, 0, 200, 77, 128, 63]),
    (256, 256, [0, 0, 5]), (768, 768, [97]), (255, 129, [4097]), (1, 300, [130]), (300, 1, [130]),
    (320, 512, [300] * 9), (384, 1024, [513]),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("out,inn,counts", WGRAD)
def test_weight_grad(B, out, inn, counts, dtype):
    """Products are exact and each of at most `tokens` additions is off by one fp32 step of a
    sum that stays below the sum of magnitudes; a bf16 result is rounded once more."""
    g = gen_of(out + inn + sum(counts))
    t = sum(counts)
    ck, x = stored(B, g, t, inn)
    dy = dy_of(g, t, out, 8)
    dw = torch.full((len(counts), out, inn), 5.0, device="cuda", dtype=dtype)
    off = offsets_of(counts)
    B.weight_grad(dy, ck, dw, offsets=ints(off))
    want, mag = ref.weight_grad(dy, x, off)
    tol = (max(counts) + 2) * ref.U_F32 * mag
    ref.check(dw, want, tol + (ref.U_BF16 * (want.abs() + tol) if dtype == BF16 else 0), "dW")
    old = dw.clone()
    B.weight_grad(dy, ck, dw, offsets=ints(off), accumulate=True)
    want2 = want + old.double()
    tol2 = tol + ref.U_F32 * want2.abs()
    ref.check(dw, want2, tol2 + (ref.U_BF16 * (want2.abs() + tol2) if dtype == BF16 else 0), "dW +=")


@pytest.mark.parametrize("out,inn,counts", [(8, 16, [40000]), (300, 200, [9001]), (640, 512, [700, 3, 0, 1500]),
                                            (1024, 2048, [2049]), (2500, 1100, [777])])
def test_weight_grad_of_whole_numbers_is_exact(B, out, inn, counts):
    """Small whole numbers: every partial sum is below 2^24, so fp32 holds it exactly."""
    g = gen_of(7)
    t = sum(counts)
    ck = B.new_act8(t, inn)
    ck.q[:, :inn].copy_(torch.randint(-4, 5, (t, inn), generator=g, device="cuda"))
    ck.exps[:, :(inn + 31) // 32].copy_(torch.randint(126, 130, (t, (inn + 31) // 32), generator=g, device="cuda"))
    dy = dy_of(g, t, out)
    dy.copy_(torch.randint(-3, 4, (t, out), generator=g, device="cuda"))
    x = ref.restore(ck.q[:, :inn], ck.exps[:, :(inn + 31) // 32]).cuda()
    off = offsets_of(counts)
    dw = torch.empty(len(counts), out, inn, device="cuda")
    B.weight_grad(dy, ck, dw, offsets=ints(off))
    want, mag = ref.weight_grad(dy, x, off)
    assert float(mag.max()) < 2 ** 22          # halves included
    assert torch.equal(dw.double(), want)


def test_weight_grad_dense_views_and_empty(B):
    """A 2-D dW inside a larger buffer; no tokens at all; a stored byte 255."""
    g = gen_of(3)
    ck, x = stored(B, g, 200, 96)
    dy = dy_of(g, 200, 72)
    buf = torch.full((80, 131), 3.0, device="cuda")
    B.weight_grad(dy, ck, buf[4:76, 5:101])
    want, mag = ref.weight_grad(dy, x, [0, 200])
    ref.check(buf[4:76, 5:101], want[0], 202 * ref.U_F32 * mag[0], "dW view")
    buf[4:76, 5:101] = 3.0
    assert bool((buf == 3).all())
    dw = torch.full((72, 96), 2.0, device="cuda", dtype=BF16)
    B.weight_grad(dy[:0], ck.rows_of(0, 0), dw, accumulate=True)
    assert bool((dw == 2).all())
    B.weight_grad(dy[:0], ck.rows_of(0, 0), dw)
    assert bool((dw == 0).all())
    ck.exps[17, 1] = 255                       # a group that held a NaN poisons its columns only
    dw = torch.zeros(72, 96, device="cuda")
    B.weight_grad(dy, ck, dw)
    assert not bool(torch.isfinite(dw[:, 32:64]).any()) and not bool(torch.isnan(dw[:, :32]).any())
    assert not bool(torch.isnan(dw[:, 64:]).any())


def test_weight_grad_groups_do_not_read_each_other(B):
    """NaN tokens before, between and behind the groups, and in a neighbouring group."""
    g = gen_of(4)
    ck, x = stored(B, g, 300, 160)
    dy = dy_of(g, 300, 136)
    dy[:10] = math.nan
    dy[290:] = math.inf
    dy[100:150] = math.nan                     # all of group 1
    ck.exps[:10] = 255
    ck.exps[100:150] = 255
    dw = torch.zeros(4, 136, 160, device="cuda")
    off = [10, 100, 150, 150, 290]
    B.weight_grad(dy, ck, dw, offsets=ints(off))
    for e in (0, 2, 3):
        want, mag = ref.weight_grad(dy, x, off[e:e + 2])
        ref.check(dw[e], want[0], 200 * ref.U_F32 * mag[0], f"dW of group {e}")
    assert bool(torch.isnan(dw[1]).all())


def test_weight_grad_offsets_are_clamped(B):
    g = gen_of(5)
    ck, x = stored(B, g, 100, 64)
    dy = dy_of(g, 100, 64)
    dw = torch.full((4, 64, 64), 9.0, device="cuda")
    B.weight_grad(dy, ck, dw, offsets=ints([-5, 60, 40, 90, 1 << 30]))
    want, mag = ref.weight_grad(dy, x, [0, 60])
    ref.check(dw[0], want[0], 100 * ref.U_F32 * mag[0], "clamped start")
    assert bool((dw[1] == 0).all())            # the end lies before the start
    for e, (lo, hi) in ((2, (40, 90)), (3, (90, 100))):
        want, mag = ref.weight_grad(dy, x, [lo, hi])
        ref.check(dw[e], want[0], 100 * ref.U_F32 * mag[0], f"group {e}")


@pytest.mark.parametrize("out,inn,groups,top", [
    (320, 512, 64, 700),       # a layer's experts: runs of tiles of equal work
    (40, 24, 200, 90),         # more groups than are weighed
    (384, 256, 90, 520), (128, 520, 128, 70), (700, 260, 33, 400), (64, 64, 129, 1)])
def test_weight_grad_of_many_ragged_groups_is_exact(B, out, inn, groups, top):
    """Whole numbers again, so every tile height and every way to deal the tiles gives the same
    bits; a quarter of the groups is empty, the first and the last among them."""
    g = gen_of(groups)
    counts = torch.randint(0, top + 1, (groups,), generator=g, device="cuda").tolist()
    counts = [0 if i % 4 == 0 or i == groups - 1 else c for i, c in enumerate(counts)]
    t = max(1, sum(counts))
    ck = B.new_act8(t, inn)
    ck.q[:, :inn].copy_(torch.randint(-4, 5, (t, inn), generator=g, device="cuda"))
    ck.exps.fill_(127)
    dy = dy_of(g, t, out)
    dy.copy_(torch.randint(-3, 4, (t, out), generator=g, device="cuda"))
    off = offsets_of(counts)
    want, _ = ref.weight_grad(dy, ck.q[:, :inn], off)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = torch.full((groups, out, inn), 9.0, device="cuda")
    plan = B.WeightGradPlan(dy, ck, dw, offsets=ints(off), status=status)
    for _ in range(40):                        # again and again: copies land in another order each time
        plan.apply()
    assert torch.equal(dw.double(), want) and int(status) == 0
    B.weight_grad(dy, ck, dw, offsets=ints(off), accumulate=True)
    assert torch.equal(dw.double(), 2 * want)


def test_weight_grad_dense_of_each_tile_height_is_exact(B):
    """One tile row of 384, 256 and 128, over many tiles along `in`, many times over."""
    g = gen_of(31)
    for out, inn, tokens in ((384, 15360, 512), (256, 12288, 700), (100, 9000, 130), (1024, 1024, 16384)):
        ck = B.new_act8(tokens, inn)
        ck.q[:, :inn].copy_(torch.randint(-2, 3, (tokens, inn), generator=g, device="cuda"))
        ck.exps.fill_(126)
        dy = dy_of(g, tokens, out)
        dy.copy_(torch.randint(-2, 3, (tokens, out), generator=g, device="cuda"))
        dw = torch.zeros(out, inn, device="cuda")
        plan = B.WeightGradPlan(dy, ck, dw)
        for _ in range(20):
            plan.apply()
        assert torch.equal(dw, dy.float().t() @ (ck.q[:, :inn].float() * 0.5))     # exact in fp32 too


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("out,inn,counts", [
    (384, 1, [130]), (384, 2563, [130, 0, 65]), (256, 12289, [70]), (768, 2309, [200]), (100, 9001, [64, 3]),
    (320, 37, [90] * 70)])
def test_weight_grad_of_columns_that_end_inside_a_warp_is_exact(B, out, inn, counts, dtype):
    """Lanes past the last column leave the stores early in every chunk of rows. Whole numbers up to
    2 * 3 * 200 * 2 in fp32, with values that bf16 holds (at most 2^8) else; every tile height."""
    g = gen_of(inn)
    t = sum(counts)
    ck = B.new_act8(t, inn)
    ck.exps.fill_(127)
    dy = dy_of(g, t, out)
    if dtype == F32:
        ck.q[:, :inn].copy_(torch.randint(-3, 4, (t, inn), generator=g, device="cuda"))
        dy.copy_(torch.randint(-2, 3, (t, out), generator=g, device="cuda"))
    else:                                       # one token in eight counts: sums of at most 26 ones
        ck.q[:, :inn].copy_(torch.randint(-1, 2, (t, inn), generator=g, device="cuda"))
        dy[::8] = torch.randint(-1, 2, (len(range(0, t, 8)), out), generator=g, device="cuda").to(BF16)
        dy[torch.arange(t, device="cuda") % 8 != 0] = 0
    off = offsets_of(counts)
    want, _ = ref.weight_grad(dy, ck.q[:, :inn], off)
    buf = torch.full((len(counts), out, inn + 3), 7.0, device="cuda", dtype=dtype)
    dw = buf[..., :inn]
    plan = B.WeightGradPlan(dy, ck, dw, offsets=ints(off))
    more = B.WeightGradPlan(dy, ck, dw, offsets=ints(off), accumulate=True)
    for _ in range(5):
        plan.apply()
        assert torch.equal(dw.double(), want)
        more.apply()
        assert torch.equal(dw.double(), 2 * want)
    assert bool((buf[..., inn:] == 7).all())


def test_weight_grad_of_a_group_that_takes_longer_than_a_wait(B):
    """One of 74 small groups has all of 400 million tokens: its tile takes one CTA pair more than a
    second, longer than the limit of a single wait. All dY but a few tokens' are zero."""
    tokens, groups = 400_000_000, 74
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 20 GB")
    ck = B.Act8(torch.ones(tokens, 16, dtype=torch.int8, device="cuda"),
                torch.full((tokens, 16), 127, dtype=torch.uint8, device="cuda"), 16)
    dy = torch.zeros(tokens, 8, dtype=BF16, device="cuda")
    dy[[0, 100_000_000, tokens - 2]] = 3.0
    dw = torch.full((groups, 8, 16), 5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = ints([0] + [tokens - 1] * (groups - 1) + [tokens])
    dy[tokens - 1] = 1.0                                        # the last group's
    B.weight_grad(dy, ck, dw, offsets=off, status=status)
    assert int(status) == 0
    assert bool((dw[0] == 9).all()) and bool((dw[1:-1] == 0).all()) and bool((dw[-1] == 1).all())


# ---------------------------------------------------------------- attention
def inputs(seed, q_len, k_len, h, g, d, pad=0, sharp=1.0):
    """q, k, v, dout as views of wider buffers."""
    gen = gen_of(seed)
    m, n = sum(q_len), sum(k_len)

    def make(t, heads, s):
        w = torch.zeros(t, heads, d + pad, device="cuda", dtype=BF16)[..., :d]
        w.copy_(randn(gen, t, heads, d) * s)
        return w
    return make(m, h, sharp), make(n, g, 1.0), make(n, g, 1.0), make(m, h, 0.1)


def both(B, q, k, v, do, q_len, k_len, causal, scale=None):
    """Forward and backward pass against the float64 forms."""
    h, d = q.shape[1], q.shape[2]
    qo, ko = ints(offsets_of(q_len)), ints(offsets_of(k_len))
    s_max = torch.full((h,), -math.inf, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = B.attention_forward(q, k, v, q_offsets=qo, k_offsets=ko, causal=causal, scale=scale,
                                 s_max=s_max, status=status)
    dq, dk, dv = B.attention_backward(do, q, k, v, o, lse, q_offsets=qo, k_offsets=ko, causal=causal,
                                      scale=scale, status=status)
    assert int(status) == 0
    want, tol = ref.attention(q, k, v, q_len, k_len, causal, scale or d ** -0.5, do, o, lse)
    ref.check(o, want["o"], tol["o"], "o")
    ref.check(lse, want["lse"], tol["lse"], "lse")
    ref.check(s_max, want["s_max"], torch.as_tensor(tol["s_max"]), "s_max")
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(t, want[n], tol[n], n)
    return o, lse, s_max, dq, dk, dv


ATTN = [
    # q lengths, k lengths, heads, kv heads, head_dim
    ([1], [1], 1, 1, 64), ([1, 17, 130], None, 2, 2, 128), ([128], None, 1, 1, 128), ([127, 129], None, 2, 1, 64),
    ([256], None, 2, 1, 128), ([257], None, 1, 1, 64), ([0, 5, 0, 300, 0], None, 3, 1, 128), ([400], None, 4, 2, 8),
    ([200, 63], None, 2, 1, 40), ([65, 300], None, 4, 4, 96), ([64], [500], 2, 1, 128), ([500], [64], 2, 1, 64),
    ([3, 0, 7, 200], [0, 9, 130, 1], 2, 2, 128), ([1, 1, 1], [700, 128, 129], 4, 1, 64), ([1000], None, 1, 1, 128),
    ([640, 1, 2, 129], None, 8, 2, 128), ([130], [0], 2, 1, 64), ([0], [130], 2, 1, 64), ([1500], None, 2, 2, 72),
    ([513], [769], 3, 3, 128),
    # many heads: grids that fill the GPU take other blocks
    ([65, 300, 1, 130], None, 80, 80, 64), ([257], None, 120, 60, 40), ([3, 0, 7, 200], [0, 9, 130, 1], 100, 100, 64),
    ([64, 63], [190, 1], 128, 32, 8), ([200, 321], [64, 500], 72, 72, 128),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,k_len,h,g,d", ATTN)
def test_attention(B, q_len, k_len, h, g, d, causal):
    k_len = q_len if k_len is None else k_len
    both(B, *inputs(sum(q_len) + d, q_len, k_len, h, g, d, pad=8), q_len, k_len, causal)


def test_attention_sharp_heads_and_scale(B):
    """Logits of tens: the running maximum moves, most probabilities vanish."""
    both(B, *inputs(1, [700], [700], 2, 1, 128, sharp=6.0), [700], [700], True)
    both(B, *inputs(2, [300], [300], 2, 2, 64), [300], [300], False, scale=0.9)


def test_attention_rising_logits_move_the_maximum_every_block(B):
    q, k, v, do = inputs(3, [256], [1024], 1, 1, 64)
    ramp = torch.arange(1024, device="cuda").float()
    q[:, 0, 0], k[:, 0, 0] = 2.0, (ramp / 16).to(BF16)          # later keys score higher by far
    both(B, q, k, v, do, [256], [1024], False)
    k[:, 0, 0] = (-ramp / 16).to(BF16)
    both(B, q, k, v, do, [256], [1024], False)


def test_attention_of_packed_qkv_and_head_major_tensors(B):
    """q, k, v as views of one tensor, gradients written into views of another; and heads as
    the outer axis."""
    g = gen_of(8)
    lens = [90, 210]
    qkv = (randn(g, 300, 3, 4, 64)).to(BF16)
    dqkv = torch.full((300, 3, 4, 64), 3.0, device="cuda", dtype=BF16)
    q, k, v = qkv[:, 0], qkv[:, 1], qkv[:, 2]
    do = randn(g, 300, 4, 64).to(BF16)
    off = ints(offsets_of(lens))
    o, lse = B.attention_forward(q, k, v, q_offsets=off, k_offsets=off)
    B.attention_backward(do, q, k, v, o, lse, dqkv[:, 0], dqkv[:, 1], dqkv[:, 2], off, off)
    want, tol = ref.attention(q, k, v, lens, lens, True, 0.125, do, o, lse)
    for i, n in enumerate(("dq", "dk", "dv")):
        ref.check(dqkv[:, i], want[n], tol[n], n)
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, do)]
    res = both(B, *hm, lens, lens, True)
    assert torch.equal(res[0], o) and torch.equal(res[3], dqkv[:, 0])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n_seq,first", [(32, 0), (33, 0), (70, 700)])
def test_attention_of_many_sequences(B, n_seq, first, causal):
    """Up to 32 sequences a block finds its tile by level, beyond by bisection; the first sequence
    may start anywhere, and rows outside every sequence stay."""
    gen = torch.Generator().manual_seed(n_seq)
    lens = torch.randint(0, 90, (n_seq,), generator=gen).tolist()
    lens[3], lens[7], lens[-1] = 300, 0, 129
    k_lens = [0 if i % 11 == 5 else n + i % 3 for i, n in enumerate(lens)]
    q, k, v, do = inputs(n_seq, lens, k_lens, 2, 1, 64)
    pad = torch.zeros(first, 2, 64, device="cuda", dtype=BF16)
    q, do = torch.cat([pad, q]), torch.cat([pad, do])
    k, v = torch.cat([pad[:, :1], k]), torch.cat([pad[:, :1], v])
    qo, ko = ints(offsets_of(lens, first)), ints(offsets_of(k_lens, first))
    o = torch.full_like(q, 4.0)
    lse = torch.full((2, q.shape[0]), 4.0, device="cuda")
    grads = [torch.full_like(t, 4.0) for t in (q, k, v)]
    B.attention_forward(q, k, v, o, lse, qo, ko, causal=causal)
    B.attention_backward(do, q, k, v, o, lse, *grads, qo, ko, causal=causal)
    want, tol = ref.attention(q[first:], k[first:], v[first:], lens, k_lens, causal, 0.125, do[first:], o[first:],
                              lse[:, first:])
    ref.check(o[first:], want["o"], tol["o"], "o")
    ref.check(lse[:, first:], want["lse"], tol["lse"], "lse")
    for n, t in zip(("dq", "dk", "dv"), grads):
        ref.check(t[first:], want[n], tol[n], n)
    assert all(bool((t[:first] == 4).all()) for t in [o, *grads]) and bool((lse[:, :first] == 4).all())


def test_attention_on_two_streams_at_once(B):
    """Two plans on two streams, again and again, each with its own workspace: the bits of a call
    alone."""
    plans, outs = [], []
    for i, d in enumerate((64, 128)):
        q, k, v, do = inputs(40 + i, [900, 300], [900, 300], 4, 2, d)
        off = ints([0, 900, 1200])
        o, lse = torch.zeros_like(q), torch.zeros(4, 1200, device="cuda")
        grads = tuple(torch.zeros_like(t) for t in (q, k, v))
        plans.append(B.AttentionPlan(q, k, v, o, lse, off, off, grads=(do, *grads)))
        plans[-1].forward()
        plans[-1].backward()
        outs.append((o, lse, *grads))
    torch.cuda.synchronize()
    alone = [[t.clone() for t in ts] for ts in outs]
    streams = [torch.cuda.Stream() for _ in plans]
    for _ in range(10):
        for p, s in zip(plans, streams):
            p.forward(stream=s)
            p.backward(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(alone, outs) for a, b in zip(x, y))


def test_attention_one_sequence_without_offsets(B):
    q, k, v, do = inputs(9, [150], [170], 4, 2, 64)
    o, lse = B.attention_forward(q, k, v, causal=True)
    grads = B.attention_backward(do, q, k, v, o, lse, causal=True)
    want, tol = ref.attention(q, k, v, [150], [170], True, 0.125, do, o, lse)
    ref.check(o, want["o"], tol["o"], "o")
    for n, t in zip(("dq", "dk", "dv"), grads):
        ref.check(t, want[n], tol[n], n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows,keys", [((13, 150), None), (None, (20, 161)), ((13, 13), None), (None, (7, 7))])
def test_attention_one_sequence_with_offsets_on_one_side(B, lib, rows, keys, causal, d):
    """Through the C call: with offsets of the rows alone the sequence has all keys, with those of
    the keys alone all rows; what lies outside is not written."""
    import ctypes
    q, k, v, do = inputs(18, [170], [190], 4, 2, d)
    (a, b), (c, e) = rows or (0, 170), keys or (0, 190)
    o, lse = torch.full_like(q, 4.0), torch.full((4, 170), 4.0, device="cuda")
    grads = [torch.full_like(t, 4.0) for t in (q, k, v)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = B.AttentionPlan(q, k, v, o, lse, causal=causal, grads=(do, *grads), status=status)
    off = ints([a, b] if rows else [c, e])
    if rows:
        plan._a.q_offsets = off.data_ptr()
    else:
        plan._a.k_offsets = off.data_ptr()
    ws, stream = plan.workspace, torch.cuda.current_stream().cuda_stream
    assert lib.muon_attention_forward(ctypes.byref(plan._a), stream) == 0
    assert lib.muon_attention_backward(ctypes.byref(plan._a), ws.data_ptr(), ws.numel(), stream) == 0
    want, tol = ref.attention(q[a:b], k[c:e], v[c:e], [b - a], [e - c], causal, d ** -0.5, do[a:b], o[a:b], lse[:, a:b])
    ref.check(o[a:b], want["o"], tol["o"], "o")
    ref.check(lse[:, a:b], want["lse"], tol["lse"], "lse")
    for n, t, (lo, hi) in zip(("dq", "dk", "dv"), grads, ((a, b), (c, e), (c, e))):
        ref.check(t[lo:hi], want[n], tol[n], n)
    for t, (lo, hi) in zip([o, lse.t(), *grads], ((a, b), (a, b), (a, b), (c, e), (c, e))):
        assert bool((t[:lo] == 4).all()) and bool((t[hi:] == 4).all())
    assert int(status) == 0


def test_attention_rows_outside_every_sequence_stay(B):
    """Rows before the first and behind the last sequence are neither read nor written, and a
    sequence of NaN leaves its neighbours alone."""
    g = gen_of(10)
    m, lens = 500, [100, 77, 131]
    off = offsets_of(lens, 13)
    q, k, v, do = (randn(g, m, 2, 64).to(BF16) for _ in range(4))
    for t in (q, k, v, do):
        t[:13] = math.nan
        t[off[-1]:] = math.nan
        t[off[1]:off[2]] = math.nan
    o = torch.full((m, 2, 64), 4.0, device="cuda", dtype=BF16)
    lse = torch.full((2, m), 4.0, device="cuda")
    grads = [torch.full((m, 2, 64), 4.0, device="cuda", dtype=BF16) for _ in range(3)]
    s_max = torch.full((2,), -math.inf, device="cuda")
    B.attention_forward(q, k, v, o, lse, ints(off), ints(off), s_max=s_max)
    B.attention_backward(do, q, k, v, o, lse, *grads, ints(off), ints(off))
    for t in [o, *grads]:
        assert bool((t[:13] == 4).all()) and bool((t[off[-1]:] == 4).all())
    assert bool((lse[:, :13] == 4).all()) and bool((lse[:, off[-1]:] == 4).all())
    best = torch.full((2,), -math.inf, dtype=torch.float64, device="cuda")
    for s in (0, 2):
        a, b = off[s], off[s + 1]
        want, tol = ref.attention(q[a:b], k[a:b], v[a:b], [b - a], [b - a], True, 0.125, do[a:b], o[a:b],
                                  lse[:, a:b])
        ref.check(o[a:b], want["o"], tol["o"], f"o of sequence {s}")
        for n, t in zip(("dq", "dk", "dv"), grads):
            ref.check(t[a:b], want[n], tol[n], f"{n} of sequence {s}")
        best = torch.maximum(best, want["s_max"])
    ref.check(s_max, best, torch.tensor(1e-4), "s_max")


def test_attention_s_max_is_raised_only(B):
    q, k, v, _ = inputs(11, [50], [50], 3, 3, 64)
    s_max = torch.tensor([-math.inf, 1e4, -1e9], device="cuda")
    B.attention_forward(q, k, v, s_max=s_max)
    want, tol = ref.attention(q, k, v, [50], [50], True, 0.125)
    assert float(s_max[1]) == 1e4
    ref.check(s_max[::2], want["s_max"][::2], torch.tensor(tol["s_max"]), "s_max")
    neg = torch.full((3,), -math.inf, device="cuda")          # every logit below zero
    B.attention_forward(q.abs(), -k.abs(), v, s_max=neg)
    want, tol = ref.attention(q.abs(), -k.abs(), v, [50], [50], True, 0.125)
    assert float(want["s_max"].max()) < 0
    ref.check(neg, want["s_max"], torch.tensor(tol["s_max"]), "negative s_max")


@pytest.mark.parametrize("d", [64, 128])
def test_attention_s_max_of_minus_zero(B, d):
    """A largest logit that underflows to -0 raises s_max from -inf and from below zero to zero, and
    no further: q.k = -2^-100 exactly, times a scale of 2^-100."""
    q, k, v, _ = inputs(19, [40], [40], 3, 1, d)
    q.zero_()
    k.zero_()
    q[..., 0], k[..., 0] = 2.0 ** -50, -(2.0 ** -50)
    s_max = torch.tensor([-math.inf, -1.0, 1e-30], device="cuda")
    B.attention_forward(q, k, v, scale=2.0 ** -100, s_max=s_max)
    assert torch.equal(s_max, torch.tensor([0.0, 0.0, 1e-30], device="cuda"))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_keys_masked_by_infinite_entries(B, d):
    """Keys whose entries make every logit -inf (with queries of one sign) count for nothing, also
    where they fill the first blocks and what follows has low logits; a row that sees no other key
    has o = 0 and lse = -inf."""
    q, k, v, _ = inputs(14, [300], [300], 2, 1, d)
    q.copy_(q.abs())
    k.copy_(-40 * k.abs())
    k[:200] = -math.inf
    s_max = torch.full((2,), -math.inf, device="cuda")
    o, lse = B.attention_forward(q, k, v, s_max=s_max)
    assert bool((o[:200] == 0).all()) and bool((lse[:, :200] == -math.inf).all())
    want, tol = ref.attention(q[200:], k[200:], v[200:], [100], [100], True, d ** -0.5)
    assert float(want["s_max"].max()) < -100
    ref.check(o[200:], want["o"], tol["o"], "o")
    ref.check(lse[:, 200:], want["lse"], tol["lse"], "lse")
    ref.check(s_max, want["s_max"], torch.as_tensor(tol["s_max"]), "s_max")


@pytest.mark.parametrize("heads,d", [(4, 128), (4, 64), (160, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_gradients_of_lone_keys_are_exactly_zero(B, heads, d, causal):
    """A row that sees one key has P = 1 whatever its logit: dQ of the row is zero, and dK gets
    nothing from it, without a rounding. Sequences of one key, and first rows of causal ones."""
    q_len, k_len = [1, 5, 130, 200, 3, 140], [1, 1, 1, 200, 6, 70]
    q, k, v, do = inputs(15, q_len, k_len, heads, heads // 2, d)
    o, _, _, dq, dk, _ = both(B, q, k, v, do, q_len, k_len, causal)
    a = b = 0
    for m, n in zip(q_len, k_len):
        seen = [min(n, i + n - m + 1) if causal else n for i in range(m)]
        for i in range(m):
            if seen[i] == 1:
                assert bool((dq[a + i] == 0).all()), (m, n, i)
        if max(seen) == 1:
            assert bool((dk[b:b + n] == 0).all()), (m, n)
        a, b = a + m, b + n
    assert bool((dq != 0).any()) and bool((dk != 0).any())


@pytest.mark.parametrize("q_len,k_len,h,g,d", [([3, 10, 60], None, 2, 2, 96), ([3], [12], 2, 1, 64), ([128], [100], 3, 3, 128)])
def test_attention_gradients_of_short_sequences_round_once(B, q_len, k_len, h, g, d):
    """Sums of one block take P and dS with 16 bits, so that dV is off by the rounding of the result
    and the fp32 sums alone: 2^-8 |dV| and an eighth of the general bound, 2^-11 of the sum of
    magnitudes (what is left of P's rounding is 2^-16 of it, the error of S about 2^-12)."""
    k_len = q_len if k_len is None else k_len
    q, k, v, do = inputs(17, q_len, k_len, h, g, d)
    qo, ko = ints(offsets_of(q_len)), ints(offsets_of(k_len))
    o, lse = B.attention_forward(q, k, v, q_offsets=qo, k_offsets=ko, causal=False)
    dq, dk, dv = B.attention_backward(do, q, k, v, o, lse, q_offsets=qo, k_offsets=ko, causal=False)
    want, tol = ref.attention(q, k, v, q_len, k_len, False, d ** -0.5, do, o, lse)
    ref.check(dv, want["dv"], ref.U_BF16 * want["dv"].abs() + tol["dv"] / 8, "dv")
    for n, t in (("dq", dq), ("dk", dk)):
        ref.check(t, want[n], tol[n], n)


@pytest.mark.parametrize("heads,d", [(2, 128), (2, 64), (160, 64)])
def test_attention_gradients_by_parts_of_the_keys(B, heads, d):
    """With o and lse of all keys, the gradients of parts of the keys (one of a single key) are the
    terms of the whole: dQ adds up, dK and dV lie side by side."""
    q, k, v, do = inputs(16, [150], [150], heads, heads, d)
    o, lse = B.attention_forward(q, k, v, causal=False)
    want, tol = ref.attention(q, k, v, [150], [150], False, d ** -0.5, do, o, lse)
    parts = [(0, 1), (1, 130), (130, 150)]
    got = [B.attention_backward(do, q, k[a:b], v[a:b], o, lse, causal=False) for a, b in parts]
    # three roundings of a part's dQ to bf16, each of a term that ref.attention bounds with the sum
    mag = sum(g[0].double().abs() for g in got)
    ref.check(sum(g[0].double() for g in got), want["dq"], tol["dq"] + ref.U_BF16 * mag, "dq")
    ref.check(torch.cat([g[1] for g in got]), want["dk"], tol["dk"], "dk")
    ref.check(torch.cat([g[2] for g in got]), want["dv"], tol["dv"], "dv")
    assert bool((got[0][1] != 0).any())


def test_attention_gradients_against_differences(B):
    """A directional difference of sum(o * dout) in float64 against the kernel's gradients."""
    lens = [70, 33]
    q, k, v, do = inputs(12, lens, lens, 4, 2, 64)
    off = ints(offsets_of(lens))
    o, lse = B.attention_forward(q, k, v, q_offsets=off, k_offsets=off)
    grads = B.attention_backward(do, q, k, v, o, lse, q_offsets=off, k_offsets=off)
    gen = gen_of(99)
    for i, t in enumerate((q, k, v)):
        r = randn(gen, *t.shape).double()
        loss = []
        for eps in (1e-4, -1e-4):
            x = [q.double(), k.double(), v.double()]
            x[i] = x[i] + eps * r
            w, _ = ref.attention(*x, lens, lens, True, 0.125)
            loss.append(float((w["o"] * do.double()).sum()))
        slope = (loss[0] - loss[1]) / 2e-4
        got = float((grads[i].double() * r).sum())
        # rounding of o (in delta), P, dS and the result: each at most 2^-8 per element, random signs
        bound = 4 * 2.0 ** -8 * float((grads[i].double().norm() * 1.0)) + 1e-6
        assert abs(got - slope) <= bound, (i, got, slope, bound)


def test_equal_calls_give_equal_bits(B):
    lens = [700, 45, 300]
    q, k, v, do = inputs(13, lens, lens, 4, 1, 128)
    off = ints(offsets_of(lens))
    first = None
    ck, _ = stored(B, gen_of(2), 3000, 200)
    dy = dy_of(gen_of(1), 3000, 100)
    for _ in range(3):
        o, lse = B.attention_forward(q, k, v, q_offsets=off, k_offsets=off)
        dw = torch.zeros(100, 200, device="cuda")
        B.weight_grad(dy, ck, dw)
        res = (o, lse, dw) + B.attention_backward(do, q, k, v, o, lse, q_offsets=off, k_offsets=off)
        if first is None:
            first = [t.clone() for t in res]
        assert all(torch.equal(a, b) for a, b in zip(first, res))


def test_offsets_past_32_bits(B):
    """A head stride and a token stride whose offsets pass 2^32 elements."""
    ld = (1 << 24) + 8
    buf = torch.empty(260 * ld, device="cuda", dtype=BF16)      # 8.7 GB
    q = buf.as_strided((260, 1, 64), (ld, 64, 1))
    g = gen_of(14)
    q.copy_(randn(g, 260, 1, 64))
    k, v = (randn(g, 260, 1, 64).to(BF16) for _ in range(2))
    o, lse = B.attention_forward(q, k, v)
    o2, lse2 = B.attention_forward(q.contiguous(), k, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dy = buf.as_strided((260, 64), (ld, 1))
    ck, x = stored(B, g, 260, 64)
    dw, dw2 = (torch.zeros(64, 64, device="cuda") for _ in range(2))
    B.weight_grad(dy, ck, dw)
    B.weight_grad(dy.contiguous(), ck, dw2)
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("tokens,heads,kv_heads,d,ld,head", [
    (200, 2, 2, 64, 64, (1 << 32) + 64),        # heads outermost
    (20000, 2, 2, 64, 64, (1 << 32) + 64),      # blocks of 64 columns
    (200, 4, 2, 128, 128, (1 << 32) + 64),      # clusters share the query heads
    (260, 2, 1, 64, (1 << 24) + 8, 64), (260, 2, 2, 128, (1 << 24) + 8, 128)])
def test_written_tensors_past_32_bits(B, tokens, heads, kv_heads, d, ld, head):
    """All tensors of both passes as interleaved views of one buffer, with strides whose offsets pass
    2^32 elements: the bits of contiguous ones, and nothing written beside them."""
    plane = tokens * d if ld < head else 2 * d                  # one tensor's share of the outer stride
    outer = max((tokens - 1) * ld, (heads - 1) * head)
    buf = torch.empty(outer + 8 * plane + tokens * d + 8, device="cuda", dtype=BF16)
    names = ("q", "k", "v", "dout", "o", "dq", "dk", "dv")
    big = {n: buf.as_strided((tokens, kv_heads if n in ("k", "v", "dk", "dv") else heads, d), (ld, head, 1), i * plane)
           for i, n in enumerate(names)}
    g = gen_of(tokens + d)
    for n in names:
        big[n].copy_(randn(g, *big[n].shape))
    small = {n: t.clone(memory_format=torch.contiguous_format) for n, t in big.items()}
    edge = buf.as_strided((heads, 8), (head, 1), 8 * plane) if ld < head else buf.as_strided((tokens, 8), (ld, 1), 8 * plane)
    edge.fill_(7.0)
    lses = []
    for t in (big, small):
        lse = torch.zeros(heads, tokens, device="cuda")
        plan = B.AttentionPlan(t["q"], t["k"], t["v"], t["o"], lse, grads=(t["dout"], t["dq"], t["dk"], t["dv"]))
        plan.forward()
        plan.backward()
        lses.append(lse)
    assert torch.equal(*lses) and bool((edge == 7).all())
    for n in names:
        assert torch.equal(big[n], small[n]), n


@pytest.mark.parametrize("tokens", [100, 16384])
def test_weight_gradient_rows_and_groups_past_32_bits(B, tokens):
    """dW with rows 2^31 elements apart (whole tiles, and parts that are joined), and with groups
    2^32 apart."""
    g = gen_of(22)
    buf = torch.empty(3 * ((1 << 31) - 8) + 64, device="cuda", dtype=BF16)      # 12.9 GB
    ck, _ = stored(B, g, tokens, 40)
    dy = dy_of(g, tokens, 4)
    rows = buf.as_strided((4, 40), ((1 << 31) - 8, 1))
    groups = buf.as_strided((2, 4, 40), ((1 << 32) + 3, 40, 1), 64)
    off = ints([0, tokens // 3, tokens])
    for big, kw in ((rows, {}), (groups, dict(offsets=off))):
        small = torch.zeros(big.shape, device="cuda", dtype=BF16)
        big.zero_()
        for accumulate in (False, True):
            B.weight_grad(dy, ck, big, accumulate=accumulate, **kw)
            B.weight_grad(dy, ck, small, accumulate=accumulate, **kw)
        assert torch.equal(big, small) and bool((small != 0).any())


# ---------------------------------------------------------------- together
def test_a_training_step_from_checkpoints_to_clipped_weights(B):
    """Attention over projections of a small model: the forward pass stores its activations in
    8 bits and measures S_max, the backward pass makes the gradients from the checkpoints, and
    the Muon plan and QK-Clip read both. Every stage against its float64 form."""
    g = gen_of(20)
    tokens, hidden, h, d = 300, 256, 4, 64
    lens = [120, 180]
    off = ints(offsets_of(lens))
    x = randn(g, tokens, hidden).to(BF16)
    Ws = [randn(g, h * d, hidden) * 0.2 for _ in range(3)]
    Gs = [torch.empty(h * d, hidden, device="cuda", dtype=BF16) for _ in Ws]
    Ms = [torch.zeros_like(w) for w in Ws]
    plan = B.Plan(Ws, Gs, Ms, B.hparams(mode="muon"))
    ck = B.new_act8(tokens, hidden)
    s_max = torch.full((h,), -math.inf, device="cuda")
    clip = B.QkClipPlan([(Ws[i], n * d, d, n, 0.5) for i in range(2) for n in range(h)], s_max, tau=2.0)
    q, k, v = (((x.float() @ w.t()).to(BF16)).view(tokens, h, d) for w in Ws)
    B.act8_store([x], [ck])
    o, lse = B.attention_forward(q, k, v, q_offsets=off, k_offsets=off, s_max=s_max)
    do = randn(g, tokens, h, d).to(BF16)
    grads = B.attention_backward(do, q, k, v, o, lse, q_offsets=off, k_offsets=off)
    for i, t in enumerate(grads):
        B.weight_grad(t.reshape(tokens, h * d), ck, Gs[i])
    xr = ref.restore(ck.q, ck.exps[:, :hidden // 32]).cuda()
    want, tol = ref.attention(q, k, v, lens, lens, True, 0.125, do, o, lse)
    for i, n in enumerate(("dq", "dk", "dv")):
        ref.check(grads[i], want[n], tol[n], n)
        dw, mag = ref.weight_grad(grads[i].reshape(tokens, h * d), xr, [0, tokens])
        t = 302 * ref.U_F32 * mag
        ref.check(Gs[i], dw[0], (t + ref.U_BF16 * (dw.abs() + t))[0], f"gradient {i}")
    before = [w.clone() for w in Ws]
    clip.apply()
    gamma = (2.0 / want["s_max"]).clamp(max=1.0).sqrt()
    assert float(gamma.min()) < 0.99
    for i in range(2):
        scaled = before[i].double().view(h, d, hidden) * gamma[:, None, None]
        assert torch.allclose(Ws[i].double().view(h, d, hidden), scaled, rtol=1e-4)
    assert torch.equal(Ws[2], before[2])
    plan.step()
    torch.cuda.synchronize()
    assert plan.query_device_status() == 0
    assert all(bool(torch.isfinite(w).all()) for w in Ws) and not torch.equal(Ws[2], before[2])
    plan.close()


def test_captured_step_on_another_stream_follows_its_buffers(B):
    """Store, attention, its backward pass and the weight gradient captured on a side stream;
    a replay with other contents (and other offsets) equals eager calls on them."""
    g = gen_of(21)
    tokens, h, d, inn = 200, 2, 64, 96
    x = randn(g, tokens, inn).to(BF16)
    ck = B.new_act8(tokens, inn)
    q, k, v, do = (randn(g, tokens, h, d).to(BF16) for _ in range(4))
    o, lse = torch.zeros_like(q), torch.zeros(h, tokens, device="cuda")
    grads = [torch.zeros_like(q) for _ in range(3)]
    off = ints([0, 90, tokens])
    dw = torch.zeros(h * d, inn, device="cuda")
    att = B.AttentionPlan(q, k, v, o, lse, off, off, grads=(do, *grads))
    wg = B.WeightGradPlan(grads[0].view(tokens, h * d), ck, dw)

    def step():
        B.act8_store([x], [ck])
        att.forward()
        att.backward()
        wg.apply()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for t in (x, q, k, v, do):
        t.copy_(randn(g, *t.shape))
    off.copy_(ints([0, 131, tokens]))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (o, lse, *grads, dw, ck.q)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (o, lse, *grads, dw, ck.q)))
    want, tol = ref.attention(q, k, v, [131, 69], [131, 69], True, 0.125, do, o, lse)
    ref.check(o, want["o"], tol["o"], "o")


def test_captured_calls_that_split_their_sums(B):
    """A weight gradient split along the tokens (its second kernel is launched early), written and
    accumulated, and a backward pass whose clusters share the query heads, captured on a side stream:
    replays follow the buffers and equal eager calls bit for bit."""
    g = gen_of(23)
    tokens = 6000
    ck, _ = stored(B, g, tokens, 96)
    dy = dy_of(g, tokens, 64)
    off = ints([0, 5000, tokens])
    dws = [torch.zeros(64, 96, device="cuda"), torch.zeros(2, 64, 96, device="cuda", dtype=BF16)]
    plans = [B.WeightGradPlan(dy, ck, dws[0], accumulate=True), B.WeightGradPlan(dy, ck, dws[1], offsets=off)]
    assert all(p.workspace is not None for p in plans)          # split
    q, k, v, do = inputs(24, [500], [500], 8, 2, 128)
    o, lse = torch.zeros_like(q), torch.zeros(8, 500, device="cuda")
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    att = B.AttentionPlan(q, k, v, o, lse, grads=(do, *grads))

    def step():
        dws[0].zero_()
        for p in (plans[0], plans[1], plans[0]):
            p.apply()
        att.forward()
        att.backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        for t in (dy, q, k, v, do):
            t.copy_(randn(g, *t.shape))
        off.copy_(ints([0, 1700 * seed, tokens]))
        for t in (o, lse, *grads, *dws):
            t.fill_(9.0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, lse, *grads, *dws)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (o, lse, *grads, *dws)))
