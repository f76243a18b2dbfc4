"""Values at the ends of what the cache attention takes: very large and very small scores, queries with channels of
very different size. Each against the float64 oracle, with a bound that does not grow with the scores."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from test_gpu_kv import DT, HALF_ULP, Step, check_append, nv, tables  # noqa: F401

# (the oracle's own bound on the results, which grows with the scores, overflows here and is not used)
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:overflow encountered", "ignore:invalid value encountered")]

SIZES = [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16"), (256, "bf16"), (256, "f16")]
LOG2E = 1.4426950408889634


def set_keys(s, values):
    """Writes key value values[j] into all channels of token j of sequence 0 ([length] or [length, dim])."""
    places, page = K.key_places(s.dim), s.cache[2].shape[2] * 16
    for j, v in enumerate(values):
        pg, inner = s.table[0, j // page], (j % page) // 16
        for h in range(s.kv_heads):
            s.cache[0][pg, h, inner, places[j % 16]] = K.encode(np.broadcast_to(v, s.dim) * 2.0 ** (127 - int(s.cache[2][pg, h, inner])))
    s.load()


def absolute_values(s):
    """The same step over a cache whose values are their magnitudes: its attention is sum w |v|."""
    return [s.cache[0], s.cache[1] & 0x7F, s.cache[2], s.cache[3]]


# Softmax weights are rounded to f16 (2^-12 of each) and the sums to f32, for which 2^-11 leaves room.
@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("score", [2.0**12.1, 2.0**20.4, 2.0**24.7, 2.0**26.3, 2.0**27.9, 2.0**30.2])
@pytest.mark.parametrize("new", [1, 2, 60])
def test_large_scores_of_equal_keys(nv, dim, dt, score, new):  # noqa: F811
    """Some keys score the same, all others at least a fourteenth less: the mean of the former's values, whatever the
    scales of the blocks that they lie in, at any size of the scores (in the exponent of 2)."""
    s = Step(nv, 50, [new], [3000], 2, 1, dim, 64, dt)
    length = int(s.lengths[0])
    s.cache[2][:] = np.where(s.g.integers(0, 2, size=s.cache[2].shape) == 1, 127 - 8, 127 - 7)
    values = s.g.choice([0.5, -1.0, 0.75, 1.0, 1.625], size=length)
    values[s.g.choice(length, size=90, replace=False)] = 1.75
    values[:3] = 1.75
    set_keys(s, values)
    q = torch.full((new, 2, dim), 1.37).to(DT[dt])
    scale = score / (LOG2E * dim * 1.75 * float(q[0, 0, 0]))
    y, ref, _ = s.attend(q, scale=scale)
    mean, _ = K.attention(q.double().numpy(), absolute_values(s), s.table, s.lengths, s.offsets, scale)
    lim = 2.0**-11 * mean + HALF_ULP[dt] * np.abs(ref) + (2.0**-24 if dt == "f16" else 0.0)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= lim).all(), float((err / lim).max())


@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("score", [2.0**24.2, 2.0**25.6, 2.0**26.9, 2.0**28.5, 2.0**30.1])
@pytest.mark.parametrize("new", [1, 2, 60])
def test_large_scores_close_together(nv, dim, dt, score, new):  # noqa: F811
    """Scores a few units of their last place apart, growing and falling from tile to tile: which key is heaviest is a
    matter of rounding, but a result lies between the smallest and the largest value."""
    s = Step(nv, 51, [new], [3000], 2, 1, dim, 64, dt)
    length = int(s.lengths[0])
    s.cache[2][:] = 127 - 8
    values = np.full((length, dim), 1.75)
    values[:, 0] = s.g.choice([1.0, 1.25, 1.5, 1.75], size=length) * np.where(np.arange(length) // 256 % 2, 1, 0.5)
    set_keys(s, values)
    q = torch.full((new, 2, dim), 1.5).to(DT[dt])
    q[..., 0] = 1.5 * 2.0**-11
    y, _, _ = s.attend(q, scale=score / (LOG2E * dim * 1.75 * 1.5))
    _, v, _ = K.dense(s.cache, s.table[0], length)
    y, most, least = y.double().cpu().numpy(), v.max((0, 1)), v.min((0, 1))
    slack = (2.0**-11 + HALF_ULP[dt]) * np.abs(v).max((0, 1))
    assert np.isfinite(y).all() and (y <= most + slack).all() and (y >= least - slack).all()


@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("up,scale", [(1.0, 1e-20), (1.0, -1e-24), (1.0, 1e-38), (1.0, 0.0), (1e-22, 0.1), (1e-30, 0.1)])
def test_small_factors_of_large_keys(nv, dim, dt, new, up, scale):  # noqa: F811
    """Keys at the top of their range along the queries or against them, under factors that make the scores small."""
    if dt == "f16" and up < 1.0:
        up, scale = 2.0**-20, scale * up * 2.0**20  # the same product: f16 has no smaller queries
    s = Step(nv, 52, [new], [700], 2, 1, dim, 64, dt)
    s.cache[2][:] = 127 + 48
    set_keys(s, s.g.choice([-448.0, 448.0], size=int(s.lengths[0])) * 2.0**48)
    q = torch.full((new, 2, dim), 1.9 * up).to(DT[dt])
    _, ref, bound = s.attend(q, scale=scale)
    mean, _ = K.attention(q.double().numpy(), absolute_values(s), s.table, s.lengths, s.offsets, scale)
    assert (bound <= 2.0**-10 * mean).all()  # scores a thousandth too large would not pass
    s.check(q, scale=scale)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("up,scale", [(1e-26, 1e34), (1e-30, 1e37), (1e-34, 2e38)])
def test_small_queries(nv, dim, new, up, scale):  # noqa: F811
    """Rows whose largest query is near bf16's smallest, under a scale that makes their scores count."""
    s = Step(nv, 55, [new], [300], 2, 1, dim, 64, "bf16")
    s.cache[2][:] = 127 - 8 - int(round(np.log2(up * scale)))
    s.load()
    q = s.rows(2, up)
    _, ref, bound = s.attend(q, scale=scale)
    mean, _ = K.attention(q.double().numpy(), absolute_values(s), s.table, s.lengths, s.offsets, scale)
    assert (bound <= 0.05 * mean).all()
    s.check(q, scale=scale)


@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("new", [1, 60])
def test_large_factors_of_small_keys(nv, dim, dt, new):  # noqa: F811
    """A scale near f32's largest, whose product with log2 e is beyond it: moderate scores of small queries and keys."""
    up, e = (1e-30, -33) if dt == "bf16" else (2.0**-20, -48)
    scale = 3e38 if dt == "bf16" else 3e18
    s = Step(nv, 53, [new], [300], 2, 1, dim, 64, dt)
    s.cache[2][:] = 127 + e
    s.load()
    q = s.rows(2, up)
    _, ref, bound = s.attend(q, scale=scale)
    mean, _ = K.attention(q.double().numpy(), absolute_values(s), s.table, s.lengths, s.offsets, scale)
    assert (bound <= 0.1 * mean).all()
    s.check(q, scale=scale)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 60])
def test_large_factors_of_large_queries(nv, dim, new):  # noqa: F811
    """Queries near bf16's largest under a large scale: the factor of the products is beyond f32, the scores are not. The
    heaviest keys' mean; a key of zeros scores zero."""
    s = Step(nv, 54, [new], [700], 2, 1, dim, 64, "bf16")
    length = int(s.lengths[0])
    s.cache[2][:] = 127 - 48
    values = s.g.choice([-1.0, 0.0, 0.5], size=length)
    values[s.g.choice(length, size=20, replace=False)] = 1.75
    values[:3] = 1.75
    set_keys(s, values * 2.0**-40)
    q = torch.full((new, 2, dim), 2.0**126, dtype=torch.bfloat16)
    y, ref, _ = s.attend(q, scale=1000.0)
    mean, _ = K.attention(q.double().numpy(), absolute_values(s), s.table, s.lengths, s.offsets, 1000.0)
    lim = 2.0**-11 * mean + HALF_ULP["bf16"] * np.abs(ref)
    assert (np.abs(y.double().cpu().numpy() - ref) <= lim).all()


def query_bound(s, q, scale, kept):
    """Bound on the results where queries down to 2^-13 of a row's largest are held as they are and smaller ones to
    `kept` of it: weights in f16, sums in f32."""
    out = np.zeros(q.shape)
    for b, length in enumerate(s.lengths):
        k, v, _ = K.dense(s.cache, s.table[b], int(length))
        for i in range(int(s.new[b])):
            n = int(length - s.new[b]) + i + 1
            for h in range(s.heads):
                kh, vh, row = k[:n, h * s.kv_heads // s.heads], v[:n, h * s.kv_heads // s.heads], q[s.offsets[b] + i, h]
                big = np.abs(row).max()
                err = np.where(np.abs(row) >= big * 2.0**-13, 0.0, np.minimum(kept * big, np.abs(row)))
                w = np.exp((kh @ row) * scale - ((kh @ row) * scale).max())
                ds = abs(scale) * (np.abs(kh) @ err + np.abs(kh) @ np.abs(row) * s.dim * 2.0**-24).max()
                out[s.offsets[b] + i, h] = (np.abs(vh).T @ (w / w.sum())) * (2.0**-11 + 2 * np.expm1(ds) + n**0.5 * 2.0**-23)
    return out


@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("new", [[1], [2, 1], [60], [130]])
@pytest.mark.parametrize("outlier,ones", [(30.0, False), (1000.0, False), (1000.0, True), (8000.0, False), (8000.0, True), (60000.0, False)])
def test_queries_with_one_large_channel(nv, dim, dt, new, outlier, ones):  # noqa: F811
    """One channel of a query far larger than the rest, and no key that uses it: the others' products keep their precision,
    and down to 2^-13 of the largest (`ones`: magnitudes from 1 to 2) they lose nothing."""
    s = Step(nv, 56, new, [200] * len(new), 2, 1, dim, 32, dt)
    places = K.key_places(dim)
    s.cache[0][..., places[:, 5]] = 0
    s.load()
    q = s.rows(2)
    if ones:
        q = torch.sign(q) * (1 + torch.from_numpy(s.g.integers(0, 128, size=tuple(q.shape)) / 128.0)).to(q.dtype)
    q[..., 5] = outlier
    y, ref, _ = s.attend(q, scale=0.4)
    lim = query_bound(s, q.double().numpy(), 0.4, 2.0**-21 if dt == "bf16" else 2.0**-24) + HALF_ULP[dt] * np.abs(ref)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= lim + (2.0**-24 if dt == "f16" else 0.0)).all(), float((err / lim).max())


@pytest.mark.parametrize("new,ctx", [([90], [-26]), ([96, 2], [-32, 100]), ([40, 80], [-40, -16]), ([300], [-100]), ([150, 1], [-22, 5])])
@pytest.mark.parametrize("heads,kv_heads,dim,window", [(1, 1, 64, 0), (2, 2, 64, 30), (2, 2, 128, 0), (4, 2, 256, 0)])
def test_more_new_tokens_than_the_length(nv, new, ctx, heads, kv_heads, dim, window):  # noqa: F811
    """Rows before a sequence's first token see no key and give zeros, also where whole tiles of rows are such."""
    s = Step(nv, 57, new, ctx, heads, kv_heads, dim, 16, "bf16")
    y = s.check(s.rows(heads), window=window)
    for b, c in enumerate(ctx):
        if c < 0:
            assert (y[int(s.offsets[b]):int(s.offsets[b]) - c] == 0).all()


@pytest.mark.parametrize("new,ctx", [([3], [500]), ([1, 3], [70, 30]), ([60], [3])])
def test_any_large_bound_on_the_new_tokens(nv, new, ctx):  # noqa: F811
    """max_q beyond the tokens there are is no different from their number, whatever it is."""
    s = Step(nv, 58, new, ctx, 8, 2, 128, 32, "bf16")
    q, args, off = s.rows(8).cuda(), (s.i32(s.table), s.i32(s.lengths)), s.i32(s.offsets)
    want = nv.kv_attention(q, s.kv, *args, q_offsets=off, max_q=sum(new))
    for max_q in (2**31, 2**61, 2**62, 2**63 - 1):
        assert torch.equal(nv.kv_attention(q, s.kv, *args, q_offsets=off, max_q=max_q), want)


def check_sharp(s, q, scale=None):
    """`Step.check`, where zeros, or a mean of the values without any scores, would not pass."""
    scale = s.dim**-0.5 if scale is None else scale
    y, ref, bound = s.attend(q, scale)
    mean, _ = K.attention(np.zeros(q.shape), s.cache, s.table, s.lengths, s.offsets, scale)
    lim = bound + HALF_ULP[s.dt] * np.abs(ref) + 2.0**-24
    several = np.repeat([int(n) - int(m) > 1 for n, m in zip(s.lengths, s.new)], s.new)  # rows that see one key have no choice
    assert (np.abs(ref) > lim)[several].mean() > 0.9 and (np.abs(ref - mean) > lim)[several].mean() > 0.9
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= lim).all(), float((err / lim).max())


@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("size", ["large", "one", "small"])
def test_query_sizes_that_count(nv, dim, dt, new, size):  # noqa: F811
    """Scores near one from queries of any size: the error that is let through is a few percent of the results."""
    up = {"large": 1e4 if dt == "f16" else 1e30, "one": 1.0, "small": 2.0**-10 if dt == "f16" else 1e-30}[size]
    s = Step(nv, 59, [new], [200], 4, 2, dim, 32, dt)
    q = s.rows(4).float()
    check_sharp(s, (q * up).to(DT[dt]), scale=float(np.float32(dim**-0.5 / up)))


# A block of threads has 160 to 512 of them: beyond, a thread looks after several sequences.
@pytest.mark.parametrize("seqs", [193, 353, 513, 1100])
@pytest.mark.parametrize("heads,kv_heads,dim,dt", [(2, 1, 64, "bf16"), (12, 1, 64, "f16"), (4, 2, 128, "bf16"), (12, 1, 128, "f16"),
                                                   (2, 1, 256, "bf16"), (4, 2, 256, "f16")])
def test_single_tokens_of_many_sequences(nv, seqs, heads, kv_heads, dim, dt):  # noqa: F811
    ctx = np.random.default_rng(seqs).integers(0, 50, size=seqs)
    ctx[::7] = 0
    ctx[5] = 500
    s = Step(nv, 60, [1] * seqs, list(ctx), heads, kv_heads, dim, 16, dt)
    check_sharp(s, s.rows(heads))


@pytest.mark.parametrize("seqs", [511, 513, 1100])
@pytest.mark.parametrize("heads,kv_heads,dim,dt,new", [(12, 1, 64, "bf16", 9), (8, 1, 128, "bf16", 5), (4, 1, 256, "f16", 3)])
def test_runs_of_many_sequences(nv, seqs, heads, kv_heads, dim, dt, new):  # noqa: F811
    """Sequences of the tensor-core kernel with single tokens and idle sequences between them."""
    g = np.random.default_rng(seqs + 1)
    n = np.where(g.random(seqs) < 0.15, new, g.integers(0, 2, size=seqs))
    n[[0, seqs - 1]] = new
    s = Step(nv, 61, list(n), list(g.integers(0, 30, size=seqs)), heads, kv_heads, dim, 16, dt)
    check_sharp(s, s.rows(heads))


@pytest.mark.parametrize("seqs", [33, 513, 1100])
def test_append_of_many_sequences(nv, seqs):  # noqa: F811
    """Single tokens, idle sequences and a chunk in one call."""
    g = np.random.default_rng(seqs + 2)
    n = g.integers(0, 2, size=seqs)
    n[seqs // 2] = 70
    s = Step(nv, 62, list(n), list(g.integers(0, 60, size=seqs)), heads=2, kv_heads=1, dim=64, page=16)
    check_append(s, s.rows(1), s.rows(1), s.rows(2), *tables(256, 64), q_offsets=s.i32(s.offsets))


@pytest.mark.parametrize("dim,dt", SIZES)
@pytest.mark.parametrize("new", [[1, 1, 1], [2, 1, 60], [130]])
def test_queries_that_are_no_numbers(nv, dim, dt, new):  # noqa: F811
    """A query with an infinity or no number gives no numbers, the other queries and heads what they give without it."""
    s = Step(nv, 63, new, [70] * len(new), 4, 2, dim, 32, dt)
    q = s.rows(4)
    want = s.check(q)
    q[0, 1, 3], q[0, 2, dim - 1], q[sum(new) - 1, 0, 0] = float("nan"), float("inf"), float("-inf")
    y = nv.kv_attention(q.cuda(), s.kv, s.i32(s.table), s.i32(s.lengths), q_offsets=s.qo(), max_q=max(new))
    bad = ~torch.isfinite(q).all(-1)
    assert torch.isnan(y[bad.cuda()]).all() and torch.equal(y[~bad.cuda()], want[~bad.cuda()])
