"""tok_sample against a plain evaluation in 64 bits: the chosen token and the
number of kept ones have to be equal, log-probabilities to within a 32-bit
rounding.  Ties, rows with few tokens or none, scores far apart and all alike,
temperatures from 0 to infinity, and the refusals."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    yield torch, pkg, tok
    tok.close()


def _plain(x, temperature=1.0, min_p=0.0, top_k=0, top_p=1.0, u=0.0):
    """(pick, kept, logprob) of a row, from the definition."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or not temperature >= 0:
        return -1, 0, -np.inf
    ids = np.flatnonzero(x > -np.inf)
    if not len(ids):
        return -1, 0, -np.inf
    ids = ids[np.lexsort((ids, -x[ids]))]
    d = x[ids] - x[ids[0]]
    w = (d == 0).astype(np.float64) if temperature < 2.0**-100 else np.exp(d / temperature)
    n = len(ids)
    if min_p > 0:
        n = int((w >= min_p).sum())
    if top_k > 0:
        n = min(n, top_k)
    if not n:
        return -1, 0, -np.inf
    cum = np.cumsum(w[:n])
    if top_p < 1:
        n = int((cum < max(top_p, 0.0) * cum[-1]).sum()) + 1
    cum = cum[:n]
    u = min(u, 1 - 2.0**-24) if u >= 0 else 0.0
    at = min(int((cum <= u * cum[-1]).sum()), n - 1)
    with np.errstate(divide="ignore"):
        return int(ids[at]), n, float(np.log(w[at] / cum[-1]))


class _Rows:
    """Rows of scores with their rules, called and checked."""

    def __init__(self, env, scores, kind, pad=0, shift=0, **rules):
        self.torch, self.pkg, self.tok = env
        torch = self.torch
        self.dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]
        x = torch.as_tensor(np.asarray(scores, np.float32))
        B, V = x.shape
        store = torch.full((B * (V + pad) + shift + 8,), float("nan"), dtype=self.dtype, device="cuda")
        self.x = store[shift:shift + B * (V + pad)].view(B, V + pad)[:, :V]
        self.x.copy_(x.to(self.dtype))
        self.kind, self.rules = kind, {}
        for k, v in rules.items():
            v = np.broadcast_to(np.asarray(v, np.int32 if k == "top_k" else np.float32), (B,)).copy()
            self.rules[k] = (v, torch.from_numpy(v).cuda())
        if "random" not in self.rules:
            v = np.random.default_rng(B + V).random(B).astype(np.float32)
            self.rules["random"] = (v, torch.from_numpy(v).cuda())
        self.pick = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
        self.kept = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
        self.logprob = torch.full((B + 1,), 7.0, device="cuda")

    def args(self, **other):
        B, V = self.x.shape
        f = dict(d_scores=self.x.data_ptr(), scores_stride=self.x.stride(0) if B > 1 else V, rows=B, n_logits=V,
                 dtype={"f32": self.pkg.DTYPE_F32, "f16": self.pkg.DTYPE_F16, "bf16": self.pkg.DTYPE_BF16}[self.kind],
                 d_pick=self.pick.data_ptr(), d_kept=self.kept.data_ptr(), d_logprob=self.logprob.data_ptr())
        f.update({"d_" + k: t.data_ptr() for k, (_, t) in self.rules.items()})
        f.update(other)
        return self.pkg.SampleArgs(**f)

    def run(self, **other):
        self.tok.sample_device(self.args(**other), self.torch.cuda.current_stream().cuda_stream)

    def check(self):
        self.run()
        x = self.x.float().cpu().numpy()
        got = [t.cpu().numpy() for t in (self.pick, self.kept, self.logprob)]
        for t, guard in zip(got, (-7, -7, 7.0)):
            assert t[-1] == guard
        for b in range(len(x)):
            r = {("u" if k == "random" else k): v[b] for k, (v, _) in self.rules.items()}
            r = {k: (int(v) if k == "top_k" else float(v)) for k, v in r.items()}
            pick, kept, lp = _plain(x[b], **r)
            assert (int(got[0][b]), int(got[1][b])) == (pick, kept), (b, r, got[0][b], got[1][b], pick, kept)
            if lp == -np.inf:
                assert got[2][b] == -np.inf
            else:
                # rounded to 32 bits once; each weight within 2^-36, the sum in steps of 2^-44 of the largest
                assert abs(got[2][b] - lp) <= 2.0**-24 * abs(lp) + 2.0**-35 + x.shape[1] * 2.0**-44, (b, got[2][b], lp)


def _scores(seed, rows, n, spread=2.5, lift=8):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, n)) * spread
    for row in x:
        at = rng.integers(0, n, max(1, min(n // 8, 40)))
        row[at] += rng.exponential(size=len(at)) * lift / 4
    return x


KINDS = ["f32", "f16", "bf16"]
SIZES = [1, 2, 7, 31, 257, 1024, 1257, 4099, 9001, 50257, 70001, 131071]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", SIZES)
def test_every_rule(env, n, kind):
    B = 24
    rng = np.random.default_rng(n)
    _Rows(env, _scores(n, B, n), kind, pad=int(rng.integers(0, 9)), shift=int(rng.integers(0, 8)),
          temperature=rng.choice([0.3, 0.7, 1.0, 1.6], B), min_p=rng.choice([0.0, 0.0, 0.02, 0.2], B),
          top_k=rng.choice([0, 1, 3, 50, max(1, n // 3), n, n + 5], B), top_p=rng.choice([1.0, 0.3, 0.9, 0.99], B),
          random=rng.random(B)).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rule", [dict(), dict(top_p=0.95), dict(top_k=40), dict(min_p=0.05), dict(top_k=3000, top_p=0.9),
                                  dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0), dict(top_k=-3, top_p=2.0, min_p=-1.0)])
def test_one_rule(env, rule, kind):
    for rows, n in ((1, 33333), (3, 100257), (200, 5003)):
        _Rows(env, _scores(rows, rows, n), kind, **rule).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("temperature", [0.0, 2.0**-120, 1e-20, 1e-4, 0.05, 20.0, 1e4, 1e30, np.inf])
def test_temperatures(env, temperature, kind):
    # (flat rows: sums of equal weights, borders at whole numbers of them; steep ones: one token)
    for rules in (dict(), dict(top_p=0.7), dict(top_k=500), dict(min_p=0.5)):
        _Rows(env, _scores(5, 6, 20011), kind, temperature=temperature, **rules).check()


@pytest.mark.parametrize("kind", KINDS)
def test_random_numbers_at_their_ends(env, kind):
    u = np.array([0.0, 2.0**-149, 2.0**-24, 0.5, 1 - 2.0**-24, 1.0, 7.0, -1.0, -0.0, np.nan, np.inf, -np.inf], np.float32)
    for spread in (2.5, 0.0):
        _Rows(env, _scores(9, len(u), 3001, spread, lift=8 if spread else 0), kind, random=u, top_p=0.9).check()


@pytest.mark.parametrize("kind", KINDS)
def test_equal_scores(env, kind):
    rng = np.random.default_rng(1)
    for n in (40, 1500, 30011, 100257):
        x = np.full((8, n), -1.25)
        x[2:4] = rng.choice([0.5, 0.75, 1.0], (2, n))        # ties of thousands
        x[4, ::3] = 2.0
        x[5] = 0.0
        x[5, ::2] = -0.0                                     # the same number
        x[6, : n // 2] = -np.inf
        x[7] = rng.integers(-3, 3, n)
        for rules in (dict(), dict(top_k=max(1, n // 2 + 3)), dict(top_p=0.37), dict(top_k=max(1, n // 5), top_p=0.81)):
            _Rows(env, x, kind, **rules).check()


@pytest.mark.parametrize("kind", ["f32"])
def test_scores_next_to_one_another(env, kind):
    # more in one bin of weights than are sorted at once: neighbouring 32-bit numbers, many of them twice
    rng = np.random.default_rng(4)
    for n in (3000, 60013):
        x = np.empty((6, n), np.float32)
        x[0] = 1 + rng.integers(0, 2 * n, n) * 2.0**-23
        x[1] = 8 + rng.integers(0, 300, n) * 2.0**-20
        x[2] = -1e-3 - rng.integers(0, 50, n) * 2.0**-33
        x[3] = np.where(rng.random(n) < 0.5, 3.0, 3.0 + rng.random(n) * 1e-4)
        x[4] = rng.integers(-2, 3, n) * 1e-30
        x[5] = 1e5 + rng.integers(0, 10, n) * 2.0**-7
        for rules in (dict(), dict(top_p=0.6), dict(top_k=n // 2), dict(top_k=n // 2, top_p=0.5, min_p=1e-3)):
            _Rows(env, x, kind, **rules).check()


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_masks_left(env, kind):
    torch = env[0]
    low = float(torch.finfo({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]).min)
    far = -1e30 if kind != "f16" else -6e4
    n = 70001
    x = _scores(6, 12, n)
    few = np.random.default_rng(8).random((12, n)) < 0.001
    x[0] = -np.inf
    x[1] = np.where(few[1], x[1], -np.inf)
    x[2] = np.where(few[2], x[2], low)
    x[3] = np.where(few[3], x[3], far)
    x[4] = low
    x[5] = far
    x[6, :-1] = -np.inf
    x[7, 1:] = low
    x[8] = np.where(few[8], x[8] - 1e4, low)
    x[9, 77] = np.inf
    x[10, 99] = np.nan
    x[11] = np.where(few[11], 5000.0, x[11])
    for rules in (dict(), dict(top_k=1000), dict(top_p=0.9), dict(min_p=0.01), dict(temperature=0.0), dict(temperature=3e4)):
        _Rows(env, x, kind, **rules).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n", [(1, 100257), (3, 100257), (200, 5003), (6, 20011), (40, 70001)])
def test_min_p_that_keeps_nothing(env, rows, n, kind):
    # rows of one CTA and of many; 16-bit rows by counts and, with scores from 2^11 on, the general way
    x = _scores(rows + n, rows, n)
    for lift in (0.0, 3000.0):
        for min_p in (1 + 2.0**-23, 1.5, np.inf):
            for rules in (dict(), dict(top_k=50), dict(top_p=0.9), dict(temperature=0.0), dict(temperature=40.0, top_k=n // 2)):
                r = _Rows(env, x + lift, kind, min_p=min_p, **rules)
                r.check()
                assert (r.pick[:-1] == -1).all() and (r.kept[:-1] == 0).all() and (r.logprob[:-1] == -np.inf).all()
    _Rows(env, x, kind, min_p=np.where(np.arange(rows) % 3, 0.01, 1.5)).check()


@pytest.mark.parametrize("temperature", [1e37, 5e37, 3e38])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scores_at_both_ends_of_the_type(env, kind, temperature):
    # differences that are not finite, at temperatures that give them weight
    rng = np.random.default_rng(3)
    x = (rng.random((8, 20011)) * 2 - 1) * 3.3e38
    x[1] = rng.choice([-3.3e38, 3.3e38], 20011)
    x[2, 1000:] = -3.3e38
    for rules in (dict(), dict(top_p=0.9), dict(top_k=5000), dict(top_k=15000, top_p=0.99), dict(min_p=1e-3)):
        _Rows(env, x, kind, temperature=temperature, **rules).check()


def _borders(kind, most, temperature, seed, steps):
    """Rows of two scores near `most` and a temperature and top-p for each, such that top_p times both weights lies
    between 2^-35.9 and 2^-32 of the first weight's: what is kept is 1 where it lies below it, else 2."""
    from decimal import Decimal, getcontext
    getcontext().prec = 40
    rng = np.random.default_rng(seed)
    place = np.spacing({"f32": np.float32, "f16": np.float16}[kind](abs(most) * 0.999))
    rows = []
    while len(rows) < 60:
        t = np.float32(temperature * (0.7 + 0.6 * rng.random()))
        m = float(np.floor(most / place) * place)
        d = float(rng.integers(1, steps)) * float(place)
        w = (Decimal(-d) / Decimal(float(t))).exp()
        p = np.float32(1 / (1 + w))
        off = abs(Decimal(float(p)) * (1 + w) - 1)
        if Decimal(2) ** Decimal("-35.9") < off < Decimal(2) ** -32 and p < 1:
            rows.append((m, m - d, t, p, 1 if Decimal(float(p)) * (1 + w) < 1 else 2))
    return rows


@pytest.mark.parametrize("kind,most,temperature,steps", [("f32", 1.5e7, 1.0, 20), ("f32", 1e6, 1.0, 200), ("f32", 1e5, 1.0, 300), ("f32", 1000.0, 0.1, 1500),
                                                         ("f32", 30.0, 1e-3, 1000), ("f32", -7e4, 2.0, 500), ("f32", 3e30, 1e25, 60),
                                                         ("f16", 50.0, 0.02, 6), ("f16", 2000.0, 0.9, 5)])
def test_borders_far_from_zero(env, kind, most, temperature, steps):
    # weights are good to 2^-36 of their size, wherever the scores lie: borders farther away are met
    rows = _borders(kind, most, temperature, 1, steps)
    x = np.array([r[:2] for r in rows])
    r = _Rows(env, x, kind, temperature=[r[2] for r in rows], top_p=[r[3] for r in rows], random=0.0)
    r.run()
    assert (r.x.double().cpu().numpy() == x).all()
    assert (r.pick[:-1] == 0).all()
    assert r.kept[:-1].tolist() == [r[4] for r in rows]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_an_infinite_temperature_at_both_ends_of_the_type(env, kind):
    # every weight is 1, whatever the differences
    rng = np.random.default_rng(4)
    x = (rng.random((6, 20011)) * 2 - 1) * 3.3e38
    x[1, 1000:] = -3.3e38
    x[2, 5:] = -np.inf
    for rules in (dict(), dict(top_p=0.9), dict(top_k=700), dict(top_k=15000, top_p=0.5), dict(min_p=1.0), dict(min_p=0.5, top_p=0.3)):
        _Rows(env, x, kind, temperature=np.inf, **rules).check()


@pytest.mark.parametrize("kind", KINDS)
def test_scores_next_to_zero(env, kind):
    x = _scores(3, 6, 5003, spread=1e-9)
    x[1] = _scores(4, 1, 5003)[0]
    x[1, 4000] = 1e-12
    x[2] *= 1e-20
    _Rows(env, x, kind, top_p=0.5).check()
    _Rows(env, x, kind, temperature=1e-9, top_p=0.5).check()


def test_temperatures_that_make_no_sense(env):
    r = _Rows(env, _scores(2, 3, 100), "bf16", temperature=[-1.0, np.nan, 1.0])
    r.check()


def test_the_largest_rows(env):
    for kind in ("f32", "f16", "bf16"):
        x = _scores(1, 2, 1 << 20)
        x[1] = 0.5
        _Rows(env, x, kind, top_p=[0.9, 0.5]).check()


def test_optional_arrays_and_repeats(env):
    torch = env[0]
    r = _Rows(env, _scores(11, 40, 30001), "f32", temperature=0.9, top_p=0.97, top_k=7000)
    r.check()
    first = [t.clone() for t in (r.pick, r.kept, r.logprob)]
    for _ in range(3):
        r.run()
        assert all(torch.equal(a, b) for a, b in zip(first, (r.pick, r.kept, r.logprob)))
    r.pick.fill_(-7)
    r.run(d_kept=None, d_logprob=None)
    assert torch.equal(r.pick, first[0])
    plain = _Rows(env, _scores(11, 40, 30001), "f32")
    plain.run(d_temperature=None, d_top_k=None, d_top_p=None, d_min_p=None)
    plain.check()


def test_streams_and_graphs(env):
    torch = env[0]
    r = _Rows(env, _scores(12, 30, 50257), "bf16", temperature=0.8, top_p=0.9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        r.run()
    side.synchronize()
    want = r.pick.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.run()
    r.pick.fill_(-7)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.pick, want)
    r.rules["random"][1].copy_(torch.rand(30))   # the graph reads what the buffers hold then
    r.rules["random"][0][:] = r.rules["random"][1].cpu().numpy()
    g.replay()
    torch.cuda.synchronize()
    got = r.pick.clone()
    r.check()
    assert torch.equal(got, r.pick)


def test_refusals(env):
    torch, pkg, tok = env
    r = _Rows(env, _scores(1, 2, 64), "f32")
    bad = [dict(d_scores=None), dict(d_random=None), dict(d_pick=None), dict(dtype=3), dict(dtype=-1), dict(n_logits=0),
           dict(n_logits=(1 << 20) + 1, scores_stride=1 << 21), dict(scores_stride=63), dict(rows=1 << 27),
           dict(d_scores=r.x.data_ptr() + 2), dict(d_kept=r.kept.data_ptr() + 1), dict(d_random=r.pick.data_ptr() + 2)]
    for other in bad:
        with pytest.raises(pkg.TokError) as e:
            r.run(**other)
        assert e.value.code == pkg.TOK_EINVAL
    r.run(rows=0, d_scores=None, d_pick=None)   # nothing to do
    torch.cuda.synchronize()
    assert (r.pick == -7).all()
