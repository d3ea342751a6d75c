"""The operators between the ids and a language model, run together by
examples/constrained_decode.py: what it decodes is the grammar's, every choice
and its log-probability are those of a 64-bit evaluation of the same scores,
and the cache's blocks are all free again at the end."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("constrained_decode", os.path.join(ROOT, "examples", "constrained_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _walk(nxt, s, data):
    for b in data:
        s = int(nxt[s, b]) if s >= 0 else -1
    return s


def _bits(words, n):
    return np.unpackbits(np.ascontiguousarray(words).view(np.uint8), bitorder="little")[:n].astype(bool)


def _decoder(ex, prompts, max_new=48, block=7):
    tok = ex.bpe.Tokenizer.from_merges_file(os.path.join(ROOT, "data", "vocabs", "gpt2_code_1k.merges"), ex.bpe.PATTERN_GPT2)
    return ex.Decoder(tok, prompts, *ex.record_grammar(), max_new=max_new, block=block)


@pytest.mark.parametrize("max_new", [48, 5])
def test_decode(ex, max_new):
    import torch
    nxt, accept = ex.record_grammar()
    prompts = [b"x = 1\n", b"", b"for i in range(10):\n    print(i)\n" * 9, b"a", "héllo".encode()]
    d = _decoder(ex, prompts, max_new)
    off = d.item_off.cpu().numpy()
    ids = d.ids.cpu().numpy()
    for k, p in enumerate(prompts):   # what was encoded, seen and placed
        mine = ids[off[k]:off[k + 1]]
        assert mine.tolist() == d.tok.encode_list(p)
        assert set(np.flatnonzero(_bits(d.seen[k].cpu().numpy(), d.V))) == set(mine.tolist())
    slots = d.slot.cpu().numpy()[:off[-1]]
    assert len(set(slots.tolist())) == off[-1]
    assert torch.equal(d.cache[d.slot[:off[-1]]], d.embed[d.ids[:off[-1]].long()])
    assert int(d.n_free) == d.n_blocks - sum(-(-int(off[k + 1] - off[k]) // d.block) for k in range(d.n))
    outs = d.run()
    for out, s in zip(outs, d.states[0].cpu().tolist()):
        end = _walk(nxt, 0, out)
        assert end >= 0
        if max_new == 48:   # the longest text has 38 bytes
            assert accept[end] and s == -1
    free = d.free.cpu().numpy()
    assert int(d.n_free) == d.n_blocks and sorted(free.tolist()) == list(range(d.n_blocks))


def test_choices(ex):
    """Each step's choice against the formulas in 64 bits.  A score's error is a
    few roundings of 32 bits at |x| < 2^5 (the logits, bfloat16, are read
    exactly): a choice may differ only where two scores lie within 2^-15; the
    sum's terms have relative errors of at most 2^-17, so has the log's argument."""
    import torch
    prompts = [b"x = 1\n", b"", b"for i in range(10):\n    print(i)\n" * 3]
    d = _decoder(ex, prompts)
    d.grammar.mask_device(d.states[0].data_ptr(), None, None, d.n, d.eos, d.states[1].data_ptr(), d.V, d.mask.data_ptr(),
                          d.words, d.stream)
    d.states.reverse()
    for _ in range(30):
        mask, seen = d.mask.cpu().numpy(), d.seen.cpu().numpy()
        gen, lens = d.gen.cpu().numpy(), d.gen_len.cpu().numpy()
        alive = d.step()
        x = d.logits.float().cpu().numpy().astype(np.float64)
        assert np.abs(x).max() < 2**5
        for k in range(d.n):
            count = np.bincount(gen[k, :lens[k]], minlength=d.V)
            pen = float(d.repetition[k])
            z = x[k].copy()
            hit = (count > 0) | _bits(seen[k], d.V)
            z[hit] = np.where(z[hit] > 0, z[hit] / pen, z[hit] * pen)
            z -= float(d.frequency[k]) * count + float(d.presence[k]) * (count > 0)
            z[d.eos] += 1.5
            z[~_bits(mask[k], d.V)] = -np.inf
            top = int(d.top[k])
            if not np.isfinite(z).any():
                assert top == -1
                continue
            assert z[top] >= z.max() - 2**-15
            y = z / float(d.temperature[k])
            want = y[top] - (y.max() + np.log(np.exp(y - y.max()).sum()))
            assert abs(float(d.logprob[k]) - want) <= 2**-14
        if not alive:
            break
    assert not alive


def test_policy_gradient(ex):
    """The gradient against the change of the log-probabilities, one score moved by h both ways."""
    import torch
    d = _decoder(ex, [b"x = 1\n", b"print(1)\n"])
    d.run()
    reward = torch.tensor([1.0, -2.0], device="cuda")
    w, grad = d.policy_gradient(reward)
    assert w.shape == d.head.shape and bool(torch.isfinite(w).all()) and float(w.norm()) > 0
    g = grad.double().cpu().numpy()
    gen, seen = d.gen.cpu().numpy(), d.seen.cpu().numpy()
    moved = 0
    for i, (_, logits, mask, gen_len, pick, _) in enumerate(d.trace):
        x = logits.double().cpu().numpy()
        for k in range(d.n):
            ok = _bits(mask[k].cpu().numpy(), d.V)
            assert not g[i, k][~ok].any()
            count = np.bincount(gen[k, :int(gen_len[k])], minlength=d.V)
            hit, pen, t = (count > 0) | _bits(seen[k], d.V), float(d.repetition[k]), float(d.temperature[k])

            def logprob(x):
                z = x.copy()
                z[hit] = np.where(z[hit] > 0, z[hit] / pen, z[hit] * pen)
                z -= float(d.frequency[k]) * count + float(d.presence[k]) * (count > 0)
                z[d.eos] += 1.5
                y = np.where(ok, z, -np.inf) / t
                return y[int(pick[k])] - (y.max() + np.log(np.exp(y - y.max()).sum()))

            for v in np.flatnonzero(ok & (x[k] != 0))[:12]:
                h = 1e-5 * min(1.0, abs(x[k, v]))   # (no kink of the penalty within)
                lo, hi = x[k].copy(), x[k].copy()
                lo[v] -= h
                hi[v] += h
                want = float(reward[k]) * (logprob(hi) - logprob(lo)) / (2 * h)
                # bfloat16 rounds at 2^-9; y - lse is off by at most 2^-16 (32-bit numbers below 2^5), and so
                # is the probability, which is below 1; the differences lose 2^-52 * 2^5 of the log
                tol = 2**-8 * abs(want) + abs(float(reward[k])) * pen / t * 2**-16 + 2**-46 / h
                assert abs(g[i, k, v] - want) <= tol, (i, k, v)
                moved += abs(want) > 0.1
    assert moved > 20
