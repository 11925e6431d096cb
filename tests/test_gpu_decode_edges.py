"""Edges of the cache, attention and sampling operators on the GPU: value scales
that say nothing of what a position counts, roundings finer than the outputs',
logits masked by finite values, and the forms of the kernels that only larger
calls take.

Against the numpy forms, tokens and cache exactly, attention within bounds that
count its roundings."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_moe_expert_q8_amd as moeq8  # noqa: E402
from oracle import decode_ref as ref  # noqa: E402
from _gpu import DEV, say  # noqa: E402
from test_gpu_decode_operators import TYPES, attention_bound, check_cache, check_sample, make_cache, typed  # noqa: E402

pytestmark = pytest.mark.gpu


def half_step(x, dtype):
    """Half of the distance of neighbouring values of dtype at x."""
    return np.ldexp(torch.finfo(dtype).eps / 2, np.frexp(np.maximum(np.abs(x), 1e-30))[1] - 1)


# ---- attention: what is rounded ----------------------------------------------------

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 40])
def test_attention_bf16_outputs_are_rounded_once(n, d):
    """Within half a step of bf16 of the definition, and what fp32 sums lose.

    The scores are near 0 and all values positive, so that little else is lost: the
    rest of the bound is that of fp32 outputs, some 2^-16 of the value.  A weight
    of 11 bits would be off by up to 2^-11."""
    rng = np.random.default_rng(n + d)
    seqs, heads = 4, 24
    cache, arrays, _ = make_cache(seqs * 3, 1, 16, d, seed=n)
    arrays[2][:] = np.maximum(np.abs(arrays[2]), 1)
    cache.v.copy_(torch.from_numpy(arrays[2]))
    q, qv = typed(1e-3 * rng.standard_normal((seqs, 1, heads, d)), torch.bfloat16)
    table = rng.permutation(seqs * 3).astype(np.int32).reshape(seqs, 3)
    visible = np.full((seqs, 1), n, np.int32)
    got = moeq8.paged_attention_i8(q.to(DEV), cache, torch.from_numpy(table).to(DEV), torch.from_numpy(visible).to(DEV))
    want, sizes = ref.attention(qv, *arrays, table, visible, d ** -0.5)
    rest = attention_bound(want, sizes, torch.float32, d)
    bound = half_step(np.abs(want) + rest, torch.bfloat16) + rest
    err = np.abs(got.float().cpu().numpy() - want)
    say(f"attention of {n}, d {d}: {(err / bound).max():.3f} of the bound, {(err > bound).sum()} of {err.size} past it")
    assert (err <= bound).all()


def crafted(scores, value_scale, signs, heads, d, dtype, seqs=1, size=16, seed=0):
    """Attention over a sequence whose scores are chosen: column c has the scores
    signs[c] * scores; of seqs alike, which read the same pages.  (got, want, bound).

    A score is one product of 1 and 1 times its scale, so of the bound's terms for
    inner products nothing is left; parts below the fp16 range lose 2^-37 of the
    largest weight times its scale and code."""
    n, cols = len(scores), len(signs)
    pages = -(-n // size)
    cache, arrays, _ = make_cache(pages, 1, size, d, seed=seed)
    k, ks, v, vs = arrays
    k[:] = 0
    k[..., 0] = 1
    ks.reshape(-1)[:n], vs.reshape(-1)[:n] = scores, value_scale
    for t, a in zip(cache, arrays):
        t.copy_(torch.from_numpy(a))
    q = np.zeros((1, cols, heads, d), np.float32)
    q[..., 0] = np.asarray(signs)[None, :, None]
    table, visible = np.arange(pages, dtype=np.int32)[None], np.full((1, cols), n, np.int32)
    alike = lambda a: torch.from_numpy(np.repeat(a, seqs, 0)).to(DEV)
    got = moeq8.paged_attention_i8(alike(q).to(dtype), cache, alike(table), alike(visible), scale=1.0)
    assert torch.equal(got, got[:1].expand_as(got))
    want, sizes = ref.attention(q, *arrays, table, visible, 1.0)
    t = np.asarray(signs, np.float64)[:, None] * ks.reshape(-1)[:n].astype(np.float64)
    w = np.exp(t - t.max(1, keepdims=True))
    top = (w / w.sum(1, keepdims=True) * vs.reshape(-1)[:n]).max(1)
    with np.errstate(all="ignore"):                         # no bound for scores past what fp32 tells apart
        bound = attention_bound(want, (sizes[0], 0 * sizes[1], *sizes[2:]), dtype, d) + (n * 2.0**-37 * 127 * top)[None, :, None, None]
    return got[:1].float().cpu().numpy(), want, bound


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("heads,d,seqs", [(2, 64, 1), (20, 128, 1), (40, 64, 1), (3, 256, 1), (2, 64, 2100), (20, 64, 2100), (3, 256, 2100)])
@pytest.mark.parametrize("where", ["one", "first", "falling", "last"])
def test_attention_loud_scales_of_positions_that_do_not_count(where, heads, d, seqs, dtype):
    """Value scales far above the others' where the weight is next to nothing, seen
    before, among or after those that count; where there are many sequences a wave
    goes through many tiles."""
    rng = np.random.default_rng(7)
    n = 700
    scores, vs = rng.uniform(-1, 1, n), rng.uniform(0.005, 0.03, n)
    if where == "one":
        scores[350], vs[350] = -60, 1e12
    elif where == "first":
        scores[:64], vs[:64] = -80, 1e12
    elif where == "last":
        scores[-40:], vs[-40:] = -80, 1e12
    else:                                                   # the maximum grows a little every time, the scales fall
        scores = np.linspace(-80, 0, n)
        vs = 0.01 * np.exp(np.linspace(60, 0, n))
    got, want, bound = crafted(scores.astype(np.float32), vs.astype(np.float32), [1.0], heads, d, TYPES[dtype], seqs)
    err = np.abs(got - want)
    say(f"loud scales {where} {heads} {d} {seqs} {dtype}: {(err / bound).max():.3f} of the bound")
    assert (err <= bound).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,d", [(2, 64), (20, 64), (3, 128)])
def test_attention_a_scale_that_counts_in_one_row_alone(heads, d, dtype):
    """The loud position has all the weight of one column and none of the other's."""
    rng = np.random.default_rng(8)
    scores, vs = rng.uniform(-1, 1, 300), rng.uniform(0.005, 0.03, 300)
    scores[99], vs[99] = -70, 1e12
    got, want, bound = crafted(scores.astype(np.float32), vs.astype(np.float32), [1.0, -1.0], heads, d, TYPES[dtype])
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,d,seqs", [(2, 64, 1), (20, 128, 1), (3, 256, 2100)])
@pytest.mark.parametrize("size", [1e5, 1e8, 3e9, 1e20, 3e29])
def test_attention_scores_past_what_fp32_tells_apart(size, heads, d, seqs, dtype):
    """Scores that lie far apart however they round: the largest has all the weight, of one
    column the first of them and of the other the last.

    Inner products are held times a power of two that brings the row's largest |q| below
    2^14, so key scales, the scores here, are good below 2^128 / (2^14 127 d) = 2^99."""
    rng = np.random.default_rng(11)
    scores, vs = size * rng.uniform(-1, 1, 300), rng.uniform(0.005, 0.03, 300)
    scores[[7, 299]] = [1.5 * size, -1.6 * size]
    got, want, _ = crafted(scores.astype(np.float32), vs.astype(np.float32), [1.0, -1.0], heads, d, TYPES[dtype], seqs)
    # a weight of 1 times scale in two fp16 parts (2^-22), the product and the sum's division
    fine = np.abs(want) * 2.0**-20
    assert (np.abs(got - want) <= fine + half_step(np.abs(want) + fine, TYPES[dtype])).all()


@pytest.mark.parametrize("up,loud,scale", [(-135, 0, 2.0**134), (-140, 0, 3e41), (100, 60, 2.0**-162), (120, 70, 2.0**-192), (-100, -60, 2.0**158)])
def test_attention_factors_past_fp32(up, loud, scale):
    """Queries of 2^up, key scales of 2^loud and a factor that fp32 does not hold, for scores around 1."""
    rng = np.random.default_rng(12)
    cache, arrays, _ = make_cache(4, 1, 16, 64, seed=12)
    arrays[1][:] = np.ldexp(arrays[1], loud)
    cache.k_scale.copy_(torch.from_numpy(arrays[1]))
    table = np.arange(4, dtype=np.int32)[None]
    q = np.ldexp(rng.standard_normal((1, 1, 2, 64)).astype(np.float32), up).astype(np.float32)
    q[0, 0, 1] = 0                                          # all alike, whatever the factor
    got = moeq8.paged_attention_i8(torch.from_numpy(q).to(DEV), cache, torch.from_numpy(table).to(DEV),
                                   torch.full((1, 1), 60, dtype=torch.int32, device=DEV), scale=scale).cpu().numpy()
    want, sizes = ref.attention(q, *arrays, table, [[60]], scale)
    assert 0.05 < sizes[2][0, 0, 0] < 50
    assert (np.abs(got - want) <= attention_bound(want, sizes, torch.float32, 64)).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_scores_of_minus_infinity(dtype):
    """They have no weight; a row that has no others gives zeros, as one that sees nothing."""
    rng = np.random.default_rng(6)
    cache, arrays, _ = make_cache(4, 1, 16, 64, seed=6)
    arrays[0][..., 0] = 1 + np.abs(arrays[0][..., 0])
    arrays[0][..., 1:] = 0
    arrays[1].reshape(-1)[:40] = np.inf
    for x, a in zip(cache, arrays):
        x.copy_(torch.from_numpy(a))
    q = torch.zeros(1, 3, 2, 64, dtype=TYPES[dtype], device=DEV)
    q[..., 0] = -1.5
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    got = moeq8.paged_attention_i8(q, cache, table, torch.tensor([[40, 7, 64]], dtype=torch.int32, device=DEV)).float().cpu().numpy()
    assert not got[:, :2].any()
    arrays[1].reshape(-1)[:40] = 1e30                       # as good as -inf, where the definition has numbers
    want, sizes = ref.attention(q.float().cpu().numpy(), *arrays, [[0, 1, 2, 3]], [[40, 7, 64]], 0.125)
    some = np.full(sizes[2].shape, 64 * 1.5 * 127 * 0.03 / 8)
    bound = attention_bound(want, (sizes[0], some, some, sizes[3]), TYPES[dtype], 64)
    assert (np.abs(got - want)[:, 2] <= bound[:, 2]).all()


def test_attention_without_a_table():
    """A table of no entries: no column sees anything."""
    cache, _, _ = make_cache(2, 2, 16, 32, seed=7)
    q = torch.randn(2, 3, 4, 32, device=DEV)
    out = moeq8.paged_attention_i8(q, cache, torch.empty(2, 0, dtype=torch.int32, device=DEV),
                                   torch.full((2, 3), 9, dtype=torch.int32, device=DEV), out=torch.full_like(q, 5.0))
    assert not out.any()


def test_calls_at_the_same_time():
    """Two streams, each with its own workspaces, against calls one after another."""
    g = torch.Generator(device=DEV).manual_seed(9)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)
    cache, _, _ = make_cache(300, 2, 16, 64, seed=9)
    table = torch.randperm(300, generator=g, device=DEV).int()[None]
    q, z = [rand(1, 2, 4, 64) for _ in range(2)], [2 * rand(40, 30011) for _ in range(2)]
    visible = [torch.tensor([[4700 - 900 * i, 4800]], dtype=torch.int32, device=DEV) for i in range(2)]
    u, p = torch.rand(40, generator=g, device=DEV), torch.full((40,), 0.9, device=DEV)
    bytes_ = (moeq8.paged_attention_workspace_bytes(1, 2, 4, 2, 64, 4800), moeq8.logits_sample_workspace_bytes(40, 30011))
    spaces = [[torch.empty(n, dtype=torch.uint8, device=DEV) for n in bytes_] for _ in range(2)]
    run = lambda i: (moeq8.paged_attention_i8(q[i], cache, table, visible[i], workspace=spaces[i][0]),
                     *moeq8.logits_sample(z[i], u, top_p=p, workspace=spaces[i][1]))
    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(result, want[i]))


# ---- sampling ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [1500, 5003])
def test_sample_never_draws_what_weighs_nothing(vocab, dtype):
    """u = 0 next to logits masked with finite values: their weights are 0 in 64 bits."""
    t = TYPES[dtype]
    rng = np.random.default_rng(vocab)
    z, zv = typed(rng.standard_normal((4, vocab)), t)
    z[0, :700] = torch.finfo(t).min
    z[1, :1030] = -1e4
    z[2, :512] = -800.0
    z[3, :600] = -60.0                                      # e^-60 is something
    u = torch.zeros(4, device=DEV)
    token, logprob = moeq8.logits_sample(z.to(DEV), u)
    zv = z.float().numpy()
    for r in range(4):
        want, log = ref.sample_row(zv[r], 0.0)
        assert int(token[r]) == want and abs(float(logprob[r]) - log) <= 2.0**-23 * abs(log)
    # at a temperature under which they weigh something after all
    token, _ = moeq8.logits_sample(z[1:3].to(DEV), u[:2], temperature=torch.full((2,), 50.0, device=DEV))
    assert token.tolist() == [ref.sample_row(r, 0.0, 50.0)[0] for r in zv[1:3]]


def masked_rows(rows, vocab, kept, value, seed):
    rng = np.random.default_rng(seed)
    z = np.full((rows, vocab), value)
    z[:, 5000:5000 + kept] = 2 * rng.standard_normal((rows, kept))
    return z, rng.uniform(0, 1, rows)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kept", [1, 300, 2000, 10000, 40000])
def test_sample_masks_of_finite_values(kept, dtype):
    """Most of a vocabulary masked with a value whose weight is 0: fewer tokens, or
    segments, than k that have one.

    Weights are held to 2^-47 for this vocabulary: with rules, one below 2^-48 is 0 and
    not drawn by u = 0 either.  Those rank behind all others, so leaving them out
    changes nothing of what the rules keep of the others."""
    vocab, t = 60011, TYPES[dtype]
    for value in (-1e4, float(torch.finfo(t).min)):
        z, u = masked_rows(3, vocab, kept, value, kept)
        u[0] = 0
        zt, zv = typed(z, t)
        u = u.astype(np.float32)
        for rules in (dict(top_k=50), dict(top_k=500), dict(top_k=5000), dict(top_k=50, top_p=0.9), dict(top_k=500, min_p=0.02),
                      dict(top_k=500, top_p=0.8, min_p=0.01), dict(top_k=500, top_p=0.8, min_p=1e-25), dict(top_k=70, temperature=0.05),
                      dict(top_p=0.9), dict(min_p=0.02), dict(top_p=0.9, min_p=1e-25), dict(top_p=0.9, min_p=1e-25, top_k=20000)):
            as_f32 = {k: np.float32(v).item() if k != "top_k" else v for k, v in rules.items()}
            vectors = {k: torch.full((3,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device=DEV) for k, v in rules.items()}
            token, logprob = moeq8.logits_sample(zt.to(DEV), torch.from_numpy(u).to(DEV), **vectors)
            for r in range(3):
                weight = np.exp((zv[r].astype(np.float64) - zv[r].max()) / as_f32.get("temperature", 1.0))
                want, log = ref.sample_row(np.where(weight < 2.0**-48, -np.inf, zv[r]), float(u[r]), **as_f32)
                assert int(token[r]) == want, (value, rules, r)
                assert abs(float(logprob[r]) - log) <= 2.0**-23 * max(abs(log), 1e-7), (value, rules, r)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rules", [dict(top_k=100), dict(top_k=100, top_p=0.9), dict(top_k=100, min_p=0.3), dict(top_k=90, top_p=0.7, min_p=0.05),
                                   dict(min_p=1e-3), dict(min_p=1e-4, top_p=0.97), dict(min_p=1e-3, top_p=0.3)],
                         ids=lambda r: "-".join(f"{k}{v}" for k, v in r.items()))
def test_sample_more_candidates_than_a_list_holds(rules, dtype):
    """A vocabulary in the order of its frequencies: the largest logits of its segments
    say little of the largest of all; and logits that nearly all pass min-p."""
    rng = np.random.default_rng(41)
    z, u = rng.standard_normal((4, 60011)), rng.uniform(0, 1, 4)
    z[0] -= np.arange(60011) / 2000
    z[1] += np.arange(60011) / 2000
    z[2] = np.round(8 * (z[2] - np.abs(np.arange(60011) - 30000) / 3000)) / 8
    z[3] *= 1.5
    check_sample(z, u, TYPES[dtype], **rules)


def test_sample_masks_of_finite_values_cost_no_more():
    """Masked with -1e4 a row takes about twice as long as masked with -inf, and not a
    selection over all of it (nine times as long)."""
    times = {}
    for value in (-1e4, -float("inf")):
        z, u = masked_rows(8, 131072, 10000, value, 1)
        z, u = torch.from_numpy(z).float().to(DEV), torch.from_numpy(u).float().to(DEV)
        k = torch.full((8,), 50, dtype=torch.int32, device=DEV)
        run = lambda: moeq8.logits_sample(z, u, top_k=k)
        run()
        taken = []
        for _ in range(5):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            for _ in range(50):
                run()
            end.record()
            end.synchronize()
            taken.append(begin.elapsed_time(end) * 20)
        times[value] = sorted(taken)[2]
    say(f"masked: {times}")
    assert times[-1e4] < 4 * times[-float("inf")]


# ---- cache -------------------------------------------------------------------------

def test_cache_arrays_that_take_turns_in_a_buffer():
    """Keys, values and their scales of each page together; outputs [token][head][k or v]."""
    pages, heads, size, d = 5, 3, 16, 48
    codes, scales = heads * size * d, heads * size * 4
    buf = torch.zeros(pages, 2 * codes + 2 * scales, dtype=torch.int8, device=DEV)
    k, v = (buf[:, i * codes:(i + 1) * codes].view(pages, heads, size, d) for i in range(2))
    ks, vs = (buf.view(torch.float32)[:, (2 * codes + i * scales) // 4:][:, :heads * size].view(pages, heads, size) for i in range(2))
    cache = moeq8.KVCacheI8(k, ks, v, vs)
    rng = np.random.default_rng(3)
    slots = rng.permutation(pages * size)[:50].astype(np.int64)
    x = rng.standard_normal((2, 50, heads, d)).astype(np.float32)
    arrays = [t.cpu().numpy().copy() for t in cache]
    moeq8.kv_cache_write_i8(*(torch.from_numpy(y).to(DEV) for y in x), cache, torch.from_numpy(slots).to(DEV))
    for i in range(2):
        ref.cache_write(arrays[2 * i], arrays[2 * i + 1], x[i], slots)
    assert all(np.array_equal(t.cpu().numpy(), a) for t, a in zip(cache, arrays))
    out = torch.zeros(50, heads, 2, d, device=DEV)
    moeq8.kv_cache_read_i8(cache, torch.from_numpy(slots).to(DEV), k_out=out[:, :, 0], v_out=out[:, :, 1])
    for i in range(2):
        assert np.array_equal(out[:, :, i].cpu().numpy(), ref.cache_read(arrays[2 * i], arrays[2 * i + 1], slots))
    with pytest.raises(moeq8.MoeQ8Error):
        moeq8.kv_cache_read_i8(cache, torch.from_numpy(slots[:40]).to(DEV), k_out=out[:40, :, 0], v_out=out[10:, :, 0])
    with pytest.raises(moeq8.MoeQ8Error):
        moeq8.kv_cache_write_i8(torch.zeros(1, heads, d, device=DEV), torch.zeros(1, heads, d, device=DEV),
                                cache._replace(v=k[1:], k=k[:-1], k_scale=ks[1:], v_scale=vs[1:]), torch.zeros(1, dtype=torch.int64, device=DEV))


# ---- the forms that larger calls take ------------------------------------------------

# Row tiles of 16, values in 64s, blocks of four waves; the lengths with one span and with several.
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("seqs,cols,heads,kv,d,longest", [
    (67, 1, 32, 8, 64, 300), (67, 1, 32, 8, 64, 1300), (67, 5, 32, 8, 64, 1300), (67, 5, 64, 8, 64, 1300),
    (67, 1, 32, 8, 128, 300), (67, 1, 32, 8, 128, 1300), (67, 3, 64, 8, 128, 1300), (9, 5, 64, 8, 128, 1300),
    (67, 8, 8, 8, 80, 700), (67, 1, 16, 8, 256, 1300), (40, 8, 32, 8, 256, 700), (33, 8, 64, 8, 128, 900)])
def test_attention_batches(seqs, cols, heads, kv, d, longest, dtype):
    rng = np.random.default_rng(seqs + cols + d)
    size, t = 16, TYPES[dtype]
    lengths = rng.integers(1, longest + 1, seqs)
    lengths[[0, 5]], lengths[[1, 7]], lengths[2], lengths[-1] = 0, longest, 1, longest - 1
    count = -(-lengths // size)
    pages = int(count.sum()) + 2
    g = torch.Generator(device=DEV).manual_seed(seqs)
    codes = lambda: torch.randint(-127, 128, (pages, kv, size, d), generator=g, device=DEV, dtype=torch.int8)
    scale = lambda: 0.005 + 0.025 * torch.rand((pages, kv, size), generator=g, device=DEV)
    cache = moeq8.KVCacheI8(codes(), scale(), codes(), scale())
    free, table = rng.permutation(pages).astype(np.int32), np.full((seqs, int(count.max()) + 1), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(count)])
    for s in range(seqs):
        table[s, :count[s]] = free[at[s]:at[s + 1]]
    visible = np.maximum(lengths[:, None] - (cols - 1 - np.arange(cols))[None], 0).astype(np.int32)
    q, qv = typed(1.5 * rng.standard_normal((seqs, cols, heads, d)), t)
    got = moeq8.paged_attention_i8(q.to(DEV), cache, torch.from_numpy(table).to(DEV), torch.from_numpy(visible).to(DEV),
                                   max_visible=longest).float().cpu().numpy()
    arrays = [x.cpu().numpy() for x in cache]
    some = [0, 1, 2, 7, int(rng.integers(8, seqs)), seqs - 1]
    want, sizes = ref.attention(qv[some], *arrays, table[some], visible[some], d ** -0.5)
    worst = float((np.abs(got[some] - want) / attention_bound(want, sizes, t, d)).max())
    say(f"attention {seqs}x{cols}x{longest} heads {heads}/{kv} d {d} {dtype}: {worst:.3f} of the bound")
    assert worst <= 1.0 and not got[[0, 5]].any()
    assert np.isfinite(got).all()
    # each sequence as it comes out in a smaller call of the same split, whose blocks lie elsewhere
    whole = torch.from_numpy(got)
    half = moeq8.paged_attention_i8(q[1:].to(DEV), cache, torch.from_numpy(table[1:]).to(DEV),
                                    torch.from_numpy(visible[1:]).to(DEV), max_visible=longest).float().cpu()
    near = torch.from_numpy(2 * attention_bound(got[1:].astype(np.float64), (np.full(got[1:].shape, 4.0), *(
        np.full(got[1:].shape[:3], float(x.max())) for x in sizes[1:])), t, d))
    assert ((whole[1:] - half).abs() <= near).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("tokens,heads,d", [(8201, 8, 128), (16391, 8, 64), (4099, 8, 256), (5501, 6, 176), (32773, 4, 48),
                                            (32771, 8, 32), (65541, 8, 16)])
def test_cache_rows_of_a_long_prefix(tokens, heads, d, dtype):
    check_cache(tokens, heads, d, 64, TYPES[dtype], special=True, seed=tokens)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", [(1700, 5003), (1000, 9001), (4100, 2000)])
def test_sample_large_batches(rows, vocab, dtype):
    """Some rows as the definition has them, and all as in smaller batches."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)
    z = (2 * torch.randn(rows, vocab, generator=g, device=DEV)).to(TYPES[dtype])
    z[3::50, vocab // 3:] = -float("inf")
    u = rand(rows)
    some = lambda x, off: torch.where(rand(rows) < 0.5, x, off)
    rules = dict(temperature=(0.3 + rand(rows)) * (rand(rows) > 0.05), top_k=some((rand(rows) * 700).int(), 0).int(),
                 top_p=some(0.3 + 0.69 * rand(rows), 1.0), min_p=some(0.2 * rand(rows), 0.0))
    token, logprob = moeq8.logits_sample(z, u, **rules)
    plain, _ = moeq8.logits_sample(z, u)
    for at in range(0, rows, 300):
        part = slice(at, min(at + 300, rows))
        t, l = moeq8.logits_sample(z[part], u[part], **{k: v[part] for k, v in rules.items()})
        assert torch.equal(t, token[part]) and torch.equal(l, logprob[part])
        assert torch.equal(moeq8.logits_sample(z[part], u[part])[0], plain[part])
    host = z.float().cpu().numpy()
    for r in [0, 3, 53, rows - 1, *np.random.default_rng(1).integers(0, rows, 20)]:
        want, log = ref.sample_row(host[r], float(u[r]), *(rules[k][r].item() for k in ("temperature", "top_k", "top_p", "min_p")))
        assert int(token[r]) == want and abs(float(logprob[r]) - log) <= 2.0**-23 * max(abs(log), 1e-7)
        assert int(plain[r]) == ref.sample_row(host[r], float(u[r]))[0]


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_over_other_orders_of_heads_and_columns(dtype):
    """Queries and outputs [seqs][heads][cols], and rows of a projection with the keys behind them."""
    rng = np.random.default_rng(5)
    seqs, cols, heads, kv, d = 3, 4, 6, 2, 48
    cache, arrays, _ = make_cache(24, kv, 16, d, seed=5)
    q, qv = typed(1.5 * rng.standard_normal((seqs, cols, heads, d)), TYPES[dtype])
    table = torch.from_numpy(rng.permutation(24).astype(np.int32).reshape(seqs, 8)).to(DEV)
    visible = torch.tensor([[60, 61, 62, 63], [0, 0, 1, 2], [120, 121, 7, 128]], dtype=torch.int32, device=DEV)
    plain = moeq8.paged_attention_i8(q.to(DEV), cache, table, visible)
    want, sizes = ref.attention(qv, *arrays, table.cpu().numpy(), visible.cpu().numpy(), d ** -0.5)
    assert (np.abs(plain.float().cpu().numpy() - want) <= attention_bound(want, sizes, TYPES[dtype], d)).all()
    turned = torch.empty(seqs, heads, cols, d, dtype=q.dtype, device=DEV).transpose(1, 2)
    moeq8.paged_attention_i8(q.to(DEV).transpose(1, 2).contiguous().transpose(1, 2), cache, table, visible, out=turned)
    rows = torch.zeros(seqs * cols, (heads + 2 * kv) * d + 3, dtype=q.dtype, device=DEV)
    inside = rows[:, :heads * d].view(seqs, cols, heads, d)
    inside.copy_(q)
    assert torch.equal(turned, plain) and torch.equal(moeq8.paged_attention_i8(inside, cache, table, visible), plain)
