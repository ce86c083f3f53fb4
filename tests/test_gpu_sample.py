"""sample_tokens against its float64 oracle.

A token has to be the oracle's wherever no border of the row lies within
`slack` of the total weight.  A weight is off by at most 2^-30 of itself and by
one unit, 2^-(62 - ceil(log2 V)) of the largest; a partial sum and the total it
is compared with are both off by that much for each of at most V weights, so
slack = 2^-29 + 2 V 2^-(62 - ceil(log2 V)) / (total / largest).  Rows nearer
than that are not compared; they have to be few.  probs are fp32 quotients of
such weights: a weight's table entry and its product with the rest, the
reciprocal and the product round by 2^-24 each, so 4 * 2^-24 + slack < 2.5e-7
relative."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 2.5e-7


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verify_mla_gb300 as m
    m.load_library()
    return m


def settings(rng, mode, T):
    if mode == "plain":
        return dict()
    if mode == "hot":
        return dict(temperature=1.7)
    if mode == "k":
        return dict(temperature=0.7, top_k=40)
    if mode == "p":
        return dict(top_p=0.9)
    if mode == "m":
        return dict(min_p=0.1)
    if mode == "kpm":
        return dict(temperature=0.9, top_k=100, top_p=0.8, min_p=0.01)
    return dict(temperature=np.where(rng.random(T) < 0.2, 0, rng.uniform(0.05, 3, T)).astype(np.float32),
                top_k=rng.choice([0, 1, 2, 5, 50, 1000, 10 ** 9, -3], T).astype(np.int32),
                top_p=rng.choice([1.0, 0.999, 0.95, 0.5, 0.01, 0.0, 2.0], T).astype(np.float32),
                min_p=rng.choice([0.0, 0.0, 0.02, 0.3, 1.0, -1.0], T).astype(np.float32))


def dev(v):
    return torch.from_numpy(np.ascontiguousarray(v)).to(DEV) if isinstance(v, np.ndarray) else v


def run(sv, x, u, s, probs=True, **kw):
    out = sv.sample_tokens(x, dev(u), return_probs=probs, **{k: dev(v) for k, v in s.items()}, **kw)
    torch.cuda.synchronize()
    return (out[0].cpu().numpy(), out[1].cpu().numpy()) if probs else out.cpu().numpy()


def check(sv, x, u, s):
    """x: a tensor of logits on the device."""
    T, V = x.shape
    ref_t, ref_p, gap, weight = oracle.ref_sample_tokens(x.float().cpu().numpy(), u, **s)
    slack = 2.0 ** -29 + 2.0 * V * 2.0 ** -(62 - int(np.ceil(np.log2(V)))) / weight
    tok, p = run(sv, x, u, s)
    only = run(sv, x, u, s, probs=False)
    assert np.array_equal(tok, only)
    sure = gap > slack
    assert np.count_nonzero(~sure) <= 1 + T // 50, gap
    assert np.array_equal(tok[sure], ref_t[sure]), (np.flatnonzero(tok != ref_t), gap[tok != ref_t])
    assert np.array_equal(p[sure] > 0, ref_p[sure] > 0)
    assert np.all(np.abs(p[sure] - ref_p[sure]) <= REL * ref_p[sure]), np.max(np.abs(p - ref_p) / np.maximum(ref_p, 1e-30))


def logits(rng, T, V, spread=2.0, peaks=8):
    x = rng.standard_normal((T, V)) * spread
    for t in range(T):
        x[t, rng.integers(0, V, peaks)] += rng.uniform(0, 8, peaks)
    return x.astype(np.float32)


MODES = ["plain", "hot", "k", "p", "m", "kpm", "mixed"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (9, 64), (4, 1000), (7, 4099), (3, 32003), (2, 163840)])
def test_shapes_and_settings(sv, T, V, mode, dtype):
    rng = np.random.default_rng(V * 7 + MODES.index(mode) + T)
    x = dev(logits(rng, T, V)).to(dtype)
    check(sv, x, rng.random(T).astype(np.float32), settings(rng, mode, T))


@pytest.mark.parametrize("T", [40, 152, 400])
def test_many_rows(sv, T):
    rng = np.random.default_rng(T)
    check(sv, dev(logits(rng, T, 5000)), rng.random(T).astype(np.float32), settings(rng, "mixed", T))


@pytest.mark.parametrize("dtype,V", [(torch.float32, 500_001), (torch.bfloat16, 1_000_003), (torch.float32, 1 << 22)])
def test_rows_beyond_shared_memory(sv, dtype, V):
    rng = np.random.default_rng(V)
    x = dev(logits(rng, 2, V)).to(dtype)
    for mode in ("kpm", "p", "plain"):
        check(sv, x, rng.random(2).astype(np.float32), settings(rng, mode, 2))


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (1, 2), (2, 3), (3, 61)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(sv, dtype, offset, pad):
    """Rows at every alignment; what lies between and around them is not read
    (it would win every draw)."""
    rng = np.random.default_rng(offset * 10 + pad)
    T, V = 6, 9001
    x = dev(logits(rng, T, V)).to(dtype)
    flat = torch.full((offset + T * (V + pad) + 8,), 8192.0, dtype=dtype, device=DEV)
    wide = flat[offset:offset + T * (V + pad)].view(T, V + pad)[:, :V]
    wide.copy_(x)
    u = rng.random(T).astype(np.float32)
    for mode in ("kpm", "plain"):
        check(sv, wide, u, settings(rng, mode, T))
    assert int((flat == 8192.0).sum().item()) == flat.numel() - T * V


def test_masks(sv):
    """-inf and NaN tokens are never drawn; rows without a finite largest logit
    draw nothing and say so, the others are not touched by it."""
    rng = np.random.default_rng(4)
    T, V = 12, 3000
    x = logits(rng, T, V)
    x[0, :] = -np.inf
    x[1, rng.random(V) < 0.9] = -np.inf
    x[2, :] = -np.inf
    x[2, 1234] = -3.5                       # one token left
    x[3, rng.random(V) < 0.5] = np.nan
    x[4, 17] = np.inf
    x[5, :] = np.finfo(np.float32).min      # all equal, the type's lowest value
    x[6, ::2] = np.finfo(np.float32).min
    x[7, :] = np.nan
    x[8, :] = 3e38
    x[9, :5] = [3e38, -3e38, 0.0, -0.0, 1e-40]
    u = rng.random(T).astype(np.float32)
    for s in (dict(), dict(top_k=10, top_p=0.9, min_p=0.01), dict(temperature=0.0), dict(top_k=2999), dict(temperature=1e30)):
        check(sv, dev(x), u, s)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        run(sv, dev(x[[0]]), u[:1], s, status=st)
        assert int(st.item()) == sv.SV_DEV_BAD_LOGITS
        st.zero_()
        run(sv, dev(x[[1, 2, 3, 5, 6, 8]]), u[:6], s, status=st)
        assert int(st.item()) == 0
    bad = np.array([np.nan, np.inf, -1.0, 0.0, -np.inf, 1e-30, 1e-20], np.float32)
    tok, p = run(sv, dev(x[[1] * 7]), u[:7], dict(temperature=bad))
    best = int(np.nanargmax(x[1]))
    assert tok.tolist() == [-1, -1] + [best] * 5 and np.all(p[:2] == 0) and np.all(p[2:, best] == 1) and np.all(p[2:].sum(1) == 1)


def test_ties(sv):
    """Equal logits in numbers: whole rows, at the k-th place, at the top-p
    border, signed zeros; greedy takes the lowest index."""
    rng = np.random.default_rng(6)
    T, V = 8, 70000
    x = np.round(rng.standard_normal((T, V)) * 2).astype(np.float32)   # a dozen distinct values
    x[1] = 0.0
    x[2, ::3] = -0.0
    x[3] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    x[4] = 1.0
    x[4, 5] = np.nextafter(np.float32(1), np.float32(2))
    u = rng.random(T).astype(np.float32)
    for s in (dict(), dict(top_k=50), dict(top_p=0.5), dict(top_k=30000, top_p=0.7), dict(min_p=1.0), dict(temperature=0.0),
              dict(top_p=0.0), dict(temperature=1e-3)):
        check(sv, dev(x), u, s)


def test_uniforms_at_the_ends(sv):
    rng = np.random.default_rng(7)
    x = logits(rng, 1, 2000)
    u = np.array([0.0, -0.0, -1.0, np.nan, 1.0, 2.0, np.inf, 1 - 2.0 ** -24, 2.0 ** -60, 1e-38], np.float32)
    tok, p = run(sv, dev(np.repeat(x, len(u), 0)), u, dict(top_k=100))
    kept = np.flatnonzero(p[0])
    assert np.all(tok[[0, 1, 2, 3, 8, 9]] == kept[0]) and np.all(tok[[4, 5, 6]] == kept[-1]) and tok[7] in kept[-3:]


@pytest.mark.parametrize("temperature", [1e-3, 0.02, 30.0, 1e4, 1e30])
def test_temperatures(sv, temperature):
    """Rows shifted by their largest logit (|x| / temperature beyond 2^13 bits)
    and not, on both sides of zero."""
    rng = np.random.default_rng(9)
    x = logits(rng, 6, 3000, spread=1.0)
    x[1] += 50
    x[2] -= 50
    x[3] *= 1000
    x[4] = x[4] * 1e-3 + 7
    for s in (dict(), dict(top_k=30), dict(top_p=0.9)):
        check(sv, dev(x), rng.random(6).astype(np.float32), dict(temperature=temperature) | s)


def test_frequencies(sv):
    """Drawn with evenly spread uniforms a token comes up in proportion to its
    probability: u runs over (i + 1/2)/n, so a count is within 1 of n p."""
    rng = np.random.default_rng(10)
    n = 4096
    x = logits(rng, 1, 700)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tok, p = run(sv, dev(x).expand(n, 700).contiguous(), u, dict(top_p=0.97))
    assert np.all(np.abs(np.bincount(tok, minlength=700) - n * p[0].astype(np.float64)) <= 1.0 + 1e-3)


def test_repeat_streams_and_graph(sv):
    """The same inputs give the same bits on any stream and in a replayed
    graph whose inputs have changed."""
    rng = np.random.default_rng(12)
    T, V = 33, 40000
    xs = [dev(logits(rng, T, V)) for _ in range(3)]
    us = [dev(rng.random(T).astype(np.float32)) for _ in range(3)]
    s = dict(temperature=0.8, top_k=60, top_p=0.9)
    want = [sv.sample_tokens(x, u, return_probs=True, **s) for x, u in zip(xs, us)]
    x, u = torch.empty_like(xs[0]), torch.empty_like(us[0])
    tokens, probs = torch.empty(T, dtype=torch.int32, device=DEV), torch.empty((T, V), device=DEV)
    torch.cuda.synchronize()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        sv.sample_tokens(x, u, tokens=tokens, probs=probs, **s)
    for i in (1, 0, 2, 2):
        x.copy_(xs[i])
        u.copy_(us[i])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, want[i][0]) and torch.equal(probs, want[i][1])


@pytest.mark.parametrize("T,V", [(1, 32773), (12, 65521), (13, 65521), (38, 40001), (76, 70001), (76, 20001), (152, 12289), (153, 9000), (320, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_work_split(sv, T, V, dtype):
    """Rows split into eight, four, two and one parts, resident or not, on both
    sides of where the split changes: the only logit of weight lies at the
    first and the last place of every part of 1/8 (and so of every other), at
    the row's ends, and the rows also carry a common distribution."""
    rng = np.random.default_rng(T + V)
    x = np.full((T, V), -80.0, np.float32)
    ends = sorted({min(max(c, 0), V - 1) for n in (1, 2, 4, 8) for i in range(n + 1) for c in
                   (lambda q: (q - 1, q))(i * ((((V + n - 1) // n) + 7) // 8 * 8))})
    at = np.array([ends[t % len(ends)] for t in range(T)])
    x[np.arange(T), at] = 3.0
    u = rng.random(T).astype(np.float32)
    for s in (dict(), dict(top_k=3), dict(top_p=0.99), dict(top_k=600, top_p=0.9), dict(min_p=0.5)):
        assert np.array_equal(run(sv, dev(x).to(dtype), u, s, probs=False), at)
    check(sv, dev(logits(rng, T, V)).to(dtype), u, settings(rng, "mixed", T))


@pytest.mark.parametrize("T", [1, 40, 160])
@pytest.mark.parametrize("kind", ["band", "few", "ends", "falling"])
def test_crowded_borders(sv, kind, T):
    """Where the estimate of a border from the counts goes wrong or the window
    around it holds more than can be listed: a band of distinct logits narrower
    than a step of the weight's grid (2^(1/512)); a band of some hundred; logits
    at both ends of one histogram bin, none between, so that its middle is a bad
    guess; a distribution in which every bin falls steeply."""
    rng = np.random.default_rng(len(kind) + T)
    V = 30011
    x = rng.standard_normal((T, V)) - 6
    if kind == "band":
        x[:, 100:28000] = 1 + 1e-3 * rng.random((T, 27900))
    elif kind == "few":
        x[:, rng.permutation(V)[:1700]] = 1 + 1e-3 * rng.random((T, 1700))
    elif kind == "ends":
        step = np.log(2) / 512
        x[:, ::2] = np.where(rng.random((T, V - V // 2)) < 0.5, 0.3, 7.6) * step + 1e-5 * rng.random((T, V - V // 2))
        x[:, 7] = 40 * step
    else:
        x = -np.abs(rng.standard_normal((T, V))) ** 0.25 * 4
    x = dev(x.astype(np.float32))
    u = rng.random(T).astype(np.float32)
    for s in (dict(top_p=0.3), dict(top_p=0.77), dict(top_k=1200, top_p=0.6), dict(top_k=9000), dict(top_k=40), dict(top_k=16000, temperature=0.5)):
        check(sv, x, u, s)


@pytest.mark.parametrize("T,V", [(2, 163840), (40, 50001), (200, 30000)])
@pytest.mark.parametrize("temperature", [0.3, 1.3])
def test_borders_among_bf16_values(sv, T, V, temperature):
    """bf16 logits lie on few values, hundreds on each, some on both sides of zero."""
    rng = np.random.default_rng(T)
    x = dev(logits(rng, T, V, peaks=24)).bfloat16()
    u = rng.random(T).astype(np.float32)
    for s in (dict(top_p=0.3), dict(top_p=0.8), dict(top_p=0.999), dict(top_k=V // 2, top_p=0.9), dict(top_k=V // 3)):
        check(sv, x, u, dict(temperature=temperature) | s)


def test_more_equal_than_candidates(sv):
    """A top-k whose last place is shared by more logits than can be ranked in
    one CTA: they are all kept."""
    rng = np.random.default_rng(21)
    for T, V in ((2, 40000), (60, 40000), (160, 3001)):
        x = logits(rng, T, V, spread=0.1, peaks=5)
        x[:, 10:1210] = 2.0
        s = dict(top_k=50)
        check(sv, dev(x), rng.random(T).astype(np.float32), s)
        assert np.all((run(sv, dev(x), rng.random(T).astype(np.float32), s)[1] > 0).sum(1) >= 1200)


@pytest.mark.parametrize("T", [1, 30, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_side_by_side(sv, T, dtype):
    """The largest logits in one stretch of the vocabulary, sorted, or falling
    with the index, so that the parts of a row say little about its k-th largest;
    and rows in which fewer logits than k have any weight."""
    rng = np.random.default_rng(24)
    V = 40003
    x = rng.standard_normal((T, V)) * 2 - 0.0003 * np.arange(V)
    x[0::3, 700:2700] += 9
    x[1::3] = np.sort(x[1::3], axis=1)
    if T > 1:
        x[2, 40:] = -200.0
    x = dev(x.astype(np.float32)).to(dtype)
    u = rng.random(T).astype(np.float32)
    for s in (dict(top_k=50, top_p=0.9), dict(top_k=250), dict(top_k=400, top_p=0.97), dict(top_k=512, min_p=0.01), dict(top_k=700, top_p=0.5)):
        check(sv, x, u, s)


def test_repeated_calls_agree(sv):
    """Nothing of a call is left for the next: calls of different shapes and
    settings in turn, on two streams at once, give each time the same bits."""
    rng = np.random.default_rng(22)
    calls = []
    for T, V, mode in ((3, 40000, "kpm"), (200, 9000, "p"), (40, 163840, "mixed"), (400, 4099, "plain")):
        calls.append((dev(logits(rng, T, V)), dev(rng.random(T).astype(np.float32)), {k: dev(v) for k, v in settings(rng, mode, T).items()}))
    want = [sv.sample_tokens(x, u, return_probs=True, **s) for x, u, s in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        got = []
        for i, (x, u, s) in enumerate(calls * 2):
            with torch.cuda.stream(streams[(i + turn) % 2]):
                got.append(sv.sample_tokens(x, u, return_probs=True, **s))
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert torch.equal(g[0], want[i % 4][0]) and torch.equal(g[1], want[i % 4][1])


def test_offsets_past_32_bits(sv):
    """Rows and distributions that begin beyond 2^31 elements, dense and by a
    stride, give what the same row gives alone."""
    T, V = 520, 1 << 22
    x = torch.empty((T, V), dtype=torch.bfloat16, device=DEV).normal_(std=2.0, generator=torch.Generator(DEV).manual_seed(1))
    u = torch.rand(T, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    for s in (dict(top_k=50), dict(min_p=0.2)):
        tok, p = sv.sample_tokens(x, u, return_probs=True, **s)
        for t in (0, T - 2, T - 1):
            one, q = sv.sample_tokens(x[t:t + 1], u[t:t + 1], return_probs=True, **s)
            assert int(one) == int(tok[t]) and torch.equal(q[0], p[t])
        del p
    far = x.view(-1)[7:].as_strided((2, 32003), (2_170_000_001, 1))
    assert torch.equal(sv.sample_tokens(far, u[:2], top_p=0.9), torch.cat([sv.sample_tokens(far[i:i + 1], u[i:i + 1], top_p=0.9) for i in (0, 1)]))


def test_many_small_rows(sv):
    """More rows than a grid dimension of 16 bits holds."""
    x = torch.randn((70001, 5), device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    u = torch.rand(70001, device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    want = x.argmax(1).int()
    assert torch.equal(sv.sample_tokens(x, u, temperature=0.0), want)
    tok, p = sv.sample_tokens(x, u, top_k=1, top_p=0.5, return_probs=True)
    hot = torch.nn.functional.one_hot(want.long(), 5).double()
    assert torch.equal(tok, want) and float((p.double() - hot).abs().max()) <= REL and int((p > 0).sum()) == 70001  # (a quotient of 1)


def test_top_k_past_32_bits(sv):
    x, u = dev(logits(np.random.default_rng(23), 3, 900)), torch.rand(3, device=DEV)
    for k, same in ((2 ** 32 + 5, 0), (2 ** 31, 0), (-2 ** 32 + 5, 0), (899, 899)):
        got, want = (sv.sample_tokens(x, u, top_k=v, return_probs=True) for v in (k, same))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(sv):
    x, u = torch.zeros((4, 100), device=DEV), torch.zeros(4, device=DEV)
    k = torch.ones(4, dtype=torch.int32, device=DEV)
    for bad in (dict(logits=x.double()), dict(logits=x.t()), dict(uniforms=u[:3]), dict(uniforms=u.double()), dict(uniforms=u.cpu()),
                dict(temperature=u.double()), dict(top_k=k.long()), dict(top_k=u), dict(top_p=u[:2]), dict(min_p=u.cpu()),
                dict(tokens=k.long()), dict(tokens=k[:2]), dict(probs=x[:, :50]), dict(probs=x.bfloat16()), dict(status=u),
                dict(logits=x[:1].expand(4, 100))):
        with pytest.raises(ValueError):
            sv.sample_tokens(**(dict(logits=x, uniforms=u) | bad))
    for bad in (dict(temperature=float("nan")), dict(top_p=float("nan")), dict(logits=x[:, :0])):
        with pytest.raises(sv.SpecVerifyError):
            sv.sample_tokens(**(dict(logits=x, uniforms=u) | bad))
    assert sv.sample_tokens(x[:0], u[:0]).shape == (0,)


def test_drafts_drawn_then_verified(sv):
    """Parallel sampling around the verify step: a prompt forked into
    continuations, drafts drawn with their distributions, sampled verification
    of them, the lengths and pages trimmed.  A draft model equal to the target
    has every draft accepted (u q(d) < p(d) for u < 1), one that never agrees
    has none."""
    rng = np.random.default_rng(14)
    torch.manual_seed(14)
    R, k, V, P, mp = 6, 3, 5000, 40, 4
    refs, table, lens = (torch.zeros(P, dtype=torch.int32, device=DEV), torch.full((R, mp), -1, dtype=torch.int32, device=DEV),
                         torch.zeros(R, dtype=torch.int32, device=DEV))
    pool = torch.randn((P, 64, 512), device=DEV).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)
    refs, table, lens = sv.kv_pages_resize(refs, table, lens, i32([100] + [0] * (R - 1)), status=status)
    refs, table, lens = sv.kv_pages_fork(pool, refs, table, lens, i32([0] * (R - 1)), i32(list(range(1, R))), status=status)
    assert lens.tolist() == [100] * R and int(refs.max().item()) == R
    refs, table, lens = sv.kv_pages_resize(refs, table, lens, lens + (k + 1), status=status)
    target = dev(logits(rng, R * (k + 1), V)).view(R, k + 1, V)
    draft = target[:, :k].contiguous()
    draft[3:] = -target[3:, :k]            # the last three requests' drafts come from another model
    drafted, q = sv.sample_tokens(draft.view(R * k, V), torch.rand(R * k, device=DEV), return_probs=True)
    u = torch.rand((R, k + 1), device=DEV).clamp(0.01, 0.98)
    accepted, nxt, kv_out = sv.spec_verify_sampled(target.view(-1, V), drafted.view(R, k), q.view(R, k, V), u, lens, k)
    p = torch.softmax(target.double(), -1)[:, :k].gather(2, drafted.view(R, k, 1).long())[..., 0]
    ratio = (p / q.view(R, k, V).gather(2, drafted.view(R, k, 1).long())[..., 0]).cpu().numpy()
    for r in range(R):
        n = 0
        while n < k and float(u[r, n]) < ratio[r, n]:
            n += 1
        assert int(accepted[r]) == n
    assert accepted[:3].tolist() == [k] * 3 and int(accepted[3:].max().item()) < k
    refs, table, lens = sv.kv_pages_resize(refs, table, lens, kv_out, status=status)
    assert torch.equal(lens, kv_out) and int(status.item()) == 0
    held = (lens.long() + 63) // 64
    assert int(refs.sum().item()) == int(held.sum().item())
