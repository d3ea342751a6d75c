"""tok_grammar_mask against a byte-by-byte walk: states and masks are whole
numbers and have to be equal.  Vocabularies with one-byte, long and shared-
prefix tokens, automata that are strict, permissive or both, duplicate states,
rows with no, one or several tokens, end tokens, and the refusals."""
import ctypes
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pkg():
    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    return pkg


def _vocab(kind):
    rng = np.random.default_rng(11)
    toks = [bytes([b]) for b in range(256)]
    if kind == "bytes":
        return toks
    seen = set(toks)
    if kind == "prefixes":  # chains of tokens that are one another's prefixes, some long
        for stem in (b"ab", b"abc", b"b", bytes([0xe4, 0xb8])):
            for n in (1, 2, 3, 4, 5, 7, 8, 9, 30, 31, 33, 255, 256, 257, 4100):
                t = (stem * n)[:n + 1]
                if t not in seen:
                    seen.add(t)
                    toks.append(t)
    n = {"prefixes": 900, "random": 5000}[kind]
    while len(toks) < n:
        t = bytes(rng.choice(list(b"abcx\"1 \xe4\xb8"), int(rng.integers(2, 9))).astype(np.uint8))
        if t not in seen:
            seen.add(t)
            toks.append(t)
    return toks


def _automaton(kind, rng):
    n = {"one": 1, "strict": 40, "loose": 7, "mixed": 60, "many": 700}[kind]
    nxt = rng.integers(0, n, (n, 256)).astype(np.int32)
    drop = {"one": 0.0, "strict": 0.97, "loose": 0.02, "many": 0.6}.get(kind)
    share = np.full((n, 1), drop) if drop is not None else rng.choice([0.0, 0.3, 0.99, 1.0], (n, 1))
    nxt[rng.random((n, 256)) < share] = -1
    if kind in ("loose", "mixed"):
        nxt[0] = 0  # a state that no byte leaves
    return nxt, (rng.random(n) < 0.5).astype(np.uint8)


def _walk(nxt, s, data):
    for b in data:
        if s < 0:
            return -1
        s = int(nxt[s, b])
    return s


def _row_state(nxt, toks, s, ids, eos):
    if not 0 <= s < len(nxt):
        return -1
    for t in ids:
        if t < 0:
            continue
        s = -1 if t == eos or t >= len(toks) or s < 0 else _walk(nxt, s, toks[t])
    return s


def _mask(nxt, accept, toks, s, eos, n_logits):
    bits = np.zeros(-(-n_logits // 32) * 32, dtype=np.uint8)
    if s >= 0:
        for t in range(min(n_logits, len(toks))):
            bits[t] = _walk(nxt, s, toks[t]) >= 0
        if 0 <= eos < n_logits:
            bits[eos] = accept[s]
    return np.packbits(bits, bitorder="little").view(np.int32)


def _run(torch, pkg, g, states, ids, off, eos, n_logits, pad=3, mask=True, out=True):
    dev = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, dtype=t)).cuda()  # noqa: E731
    words = -(-n_logits // 32)
    d_s, d_i, d_o = dev(states, np.int32), dev(ids, np.int32), dev(off, np.int64)
    d_out = torch.full((len(states) + 1,), -9, dtype=torch.int32, device="cuda")
    d_m = torch.full((len(states), words + pad), -9, dtype=torch.int32, device="cuda")
    p = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    g.mask_device(p(d_s), p(d_i), p(d_o), len(states), eos, p(d_out) if out else None, n_logits, p(d_m) if mask else None,
                  words + pad, torch.cuda.current_stream().cuda_stream)
    m = d_m.cpu().numpy()
    assert (m[:, words:] == -9).all() and d_out.cpu()[-1] == -9
    return d_out.cpu().numpy()[:-1], m[:, :words]


@pytest.mark.parametrize("vocab", ["bytes", "prefixes", "random"])
@pytest.mark.parametrize("kind", ["one", "strict", "loose", "mixed", "many"])
def test_masks(pkg, vocab, kind):
    import torch
    rng = np.random.default_rng(5)
    toks = _vocab(vocab)
    tok = pkg.Tokenizer(toks, [], pkg.PATTERN_GPT2)
    nxt, accept = _automaton(kind, rng)
    g = pkg.Grammar(tok, nxt, accept)
    V, n = len(toks), len(nxt)
    known = {}

    def mask(s, eos, n_logits):
        key = (s, eos, n_logits)
        if key not in known:
            known[key] = _mask(nxt, accept, toks, s, eos, n_logits)
        return known[key]

    # rows in random states, some outside the automaton, several in the same one; no tokens
    few = rng.integers(0, n, 6)
    for rows, eos, n_logits in ((1, -1, V), (3, V, V + 1), (300, V + 40, V + 77), (5, 3, V - 1), (2, -1, 1), (2, 0, 33)):
        states = few[rng.integers(0, 6, rows)]
        states[rng.random(rows) < 0.1] = rng.choice([-1, -5, n, n + 7])
        got, m = _run(torch, pkg, g, states, None, None, eos, n_logits)
        want = [s if 0 <= s < n else -1 for s in states]
        assert got.tolist() == want
        assert np.array_equal(m, np.stack([mask(s, eos, n_logits) for s in want])), (rows, eos, n_logits)
    # one token a row: allowed ones mostly, none, the end token, one beyond the vocabulary
    rows, eos, n_logits = 270, V, V + 2
    states = few[rng.integers(0, 6, rows)]
    ids = rng.integers(0, 256, rows)
    ids[rng.random(rows) < 0.3] = rng.integers(0, V)
    ids[:4] = -1, eos, V + 1, -7
    got, m = _run(torch, pkg, g, states, ids, None, eos, n_logits)
    want = [_row_state(nxt, toks, int(s), [int(t)], eos) for s, t in zip(states, ids)]
    assert got.tolist() == want
    assert np.array_equal(m, np.stack([mask(s, eos, n_logits) for s in want]))
    # several tokens a row, only the states; then only the masks
    lens = rng.integers(0, 4, rows)
    off = np.concatenate([[0], np.cumsum(lens)])
    ids = rng.integers(0, 256, max(1, int(off[-1])))
    got, _ = _run(torch, pkg, g, states, ids, off, eos, n_logits, mask=False)
    want = [_row_state(nxt, toks, int(s), ids[a:b].tolist(), eos) for s, a, b in zip(states, off, off[1:])]
    assert got.tolist() == want
    _, m = _run(torch, pkg, g, states, ids, off, eos, n_logits, out=False)
    assert np.array_equal(m, np.stack([mask(s, eos, n_logits) for s in want]))
    g.close()
    tok.close()


def test_every_state_of_a_trained_vocabulary(pkg):
    # sampled tokens of every state of a random automaton over 100k tokens, and the mask's count against a plain walk
    import torch
    tok = pkg.Tokenizer.from_merges_file(os.path.join(ROOT, "data", "vocabs", "cl100k_session_100k.merges"), pkg.PATTERN_CL100K)
    toks = tok.token_bytes
    rng = np.random.default_rng(2)
    n = 9
    nxt = rng.integers(0, n, (n, 256)).astype(np.int32)
    nxt[rng.random((n, 256)) < rng.choice([0.0, 0.05, 0.5, 0.98], (n, 1))] = -1
    g = pkg.Grammar(tok, nxt, np.ones(n, np.uint8))
    states = np.arange(n)
    _, m = _run(torch, pkg, g, states, None, None, len(toks), len(toks) + 1)
    bits = np.unpackbits(m.view(np.uint8), axis=1, bitorder="little")
    longest = max(map(len, toks))
    byts, lens = np.zeros((len(toks), longest), np.uint8), np.array([len(t) for t in toks])
    for k, t in enumerate(toks):
        byts[k, :len(t)] = np.frombuffer(t, np.uint8)
    for s in range(n):
        at = np.full(len(toks), s)
        for p in range(longest):
            step = (p < lens) & (at >= 0)
            at[step] = nxt[at[step], byts[step, p]]
        assert np.array_equal(bits[s, :len(toks)], (at >= 0).astype(np.uint8)), s
        assert bits[s, len(toks)] == 1 and not bits[s, len(toks) + 1:].any()
    g.close()
    tok.close()


@pytest.mark.parametrize("rows", [1, 16, 17, 40, 511, 512, 513, 1100])
@pytest.mark.parametrize("several", [False, True])
def test_states_and_masks_of_many_rows(pkg, rows, several):
    # rows in one window and in several, with states found by the masks' own kernel or before it
    import torch
    rng = np.random.default_rng(rows)
    toks = _vocab("prefixes")
    tok = pkg.Tokenizer(toks, [], pkg.PATTERN_GPT2)
    nxt, accept = _automaton("mixed", rng)
    g = pkg.Grammar(tok, nxt, accept)
    V = len(toks)
    states = rng.integers(0, len(nxt), rows)
    lens = rng.integers(0, 6, rows) if several else np.ones(rows, int)
    off = np.concatenate([[0], np.cumsum(lens)])
    ids = rng.integers(-1, 256, max(1, int(off[-1])))
    got, m = _run(torch, pkg, g, states, ids, off if several else None, V, V + 1)
    want = [_row_state(nxt, toks, int(s), ids[a:b].tolist(), V) for s, a, b in zip(states, off, off[1:])]
    assert got.tolist() == want
    masks = {s: _mask(nxt, accept, toks, s, V, V + 1) for s in set(want)}
    assert np.array_equal(m, np.stack([masks[s] for s in want]))
    g.close()
    tok.close()


def test_masks_right_after_the_load(pkg):
    # on a stream that does not wait for the default one, with work queued there: the tables are complete all the same
    import torch
    toks = _vocab("prefixes")
    V = len(toks)
    s = torch.cuda.Stream()
    states = torch.arange(700, dtype=torch.int32, device="cuda")
    words = -(-V // 32)
    busy = torch.zeros(1 << 26, device="cuda")
    for seed in range(6):
        nxt, accept = _automaton("many", np.random.default_rng(seed))
        m = torch.full((700, words), -9, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        tok = pkg.Tokenizer(toks, [], pkg.PATTERN_GPT2)
        busy.add_(1.0)
        g = pkg.Grammar(tok, nxt, accept)
        g.mask_device(states.data_ptr(), None, None, 700, -1, None, V, m.data_ptr(), words, s.cuda_stream)
        s.synchronize()
        got = m.cpu().numpy()
        for k in range(seed, 700, 97):
            assert np.array_equal(got[k], _mask(nxt, accept, toks, k, -1, V)), (seed, k)
        g.close()
        tok.close()


def test_a_grammar_may_outlive_its_tokenizer(pkg):
    # closed in either order, none keeps its automaton (31 MB here) on the device
    import torch
    nxt, acc = np.zeros((60_000, 256), np.int32), np.ones(60_000, np.uint8)
    free = []
    for k in range(8):
        tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
        g = pkg.Grammar(tok, nxt, acc)
        for x in (tok, g) if k % 2 else (g, tok):
            x.close()
        g.close()
        torch.cuda.synchronize()
        free.append(torch.cuda.mem_get_info()[0])
    assert free[-1] > free[1] - (15 << 20), free


def test_refusals(pkg):
    import torch
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    other = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    L = pkg.lib()
    nxt, acc = np.zeros((2, 256), np.int32), np.ones(2, np.uint8)
    for bad in (2, -2):
        broken = nxt.copy()
        broken[1, 255] = bad
        with pytest.raises(pkg.TokError) as e:
            pkg.Grammar(tok, broken, acc)
        assert e.value.code == pkg.TOK_EINVAL
    with pytest.raises(pkg.TokError):
        pkg.Grammar(tok, np.zeros((0, 256), np.int32), np.zeros(0, np.uint8))
    with pytest.raises(ValueError):
        pkg.Grammar(tok, nxt, np.ones(3, np.uint8))
    h = ctypes.c_void_p()
    assert L.tok_grammar_load(None, None, None, 1, ctypes.byref(h)) == pkg.TOK_EINVAL
    assert L.tok_grammar_load(tok._h, None, None, 1, ctypes.byref(h)) == pkg.TOK_EINVAL and not h.value
    # allocations that fail: the vocabulary's on the first load, then the grammar's
    for k in (1, 2):
        L.tok_debug_fail_alloc(tok._h, k)
        with pytest.raises(pkg.TokError) as e:
            pkg.Grammar(tok, nxt, acc)
        assert e.value.code == pkg.TOK_ENOMEM
        L.tok_debug_fail_alloc(tok._h, 0)
    g = pkg.Grammar(tok, nxt, acc)
    s, o = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((4,), -9, dtype=torch.int32, device="cuda")
    m = torch.full((4, 9), -9, dtype=torch.int32, device="cuda")
    good = dict(d_state=s.data_ptr(), d_ids=None, d_item_off=None, n=4, eos=256, d_state_out=o.data_ptr(), n_logits=257,
                d_mask=m.data_ptr(), mask_stride=9)
    for bad in (dict(d_state=None), dict(d_state_out=None, d_mask=None), dict(d_state_out=s.data_ptr()), dict(n_logits=0),
                dict(n_logits=(1 << 20) + 1, mask_stride=1 << 20), dict(mask_stride=8), dict(d_item_off=s.data_ptr())):
        with pytest.raises(pkg.TokError) as e:
            g.mask_device(**{**good, **bad})
        assert e.value.code == pkg.TOK_EINVAL, bad
    assert L.tok_grammar_mask(other._h, g._g, s.data_ptr(), None, None, 4, 256, o.data_ptr(), 257, m.data_ptr(), 9, None) == pkg.TOK_EINVAL
    assert L.tok_grammar_mask(None, g._g, s.data_ptr(), None, None, 4, 256, o.data_ptr(), 257, m.data_ptr(), 9, None) == pkg.TOK_EINVAL
    g.mask_device(**{**good, "n": 0})
    assert (o.cpu() == -9).all() and (m.cpu() == -9).all()
    g.mask_device(**good)
    assert o.cpu().tolist() == [0] * 4 and (m.cpu()[:, :8] == -1).all() and (m.cpu()[:, 8] == 1).all()
    g.close()
    tok.close()
    other.close()
