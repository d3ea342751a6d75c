"""What the binding hands to tok_grammar_load: next states that 32 bits hold,
and accept as 0 or 1.  The library is a stand-in, no GPU is needed."""
import numpy as np
import pytest

import exact_bpe_tokenization_utf_gb300 as pkg


class _Tok:
    """A tokenizer whose library keeps what it is given."""
    _h = 1

    def __init__(self):
        self._L = self
        self.got = None

    def _check(self, rc):
        assert rc == 0

    def tok_grammar_load(self, h, nxt, acc, n, out):
        self.got = [[nxt[k * 256 + b] for b in range(256)] for k in range(n)], [acc[k] for k in range(n)]
        return 0


def _next():
    nxt = np.full((3, 256), -1, np.int64)
    nxt[0, 65], nxt[1, 66], nxt[2, 255] = 1, 2, 0
    return nxt


@pytest.mark.parametrize("kind", [np.int8, np.int16, np.int32, np.int64, np.float64, list])
def test_next_states_arrive(kind):
    nxt, tok = _next(), _Tok()
    pkg.Grammar(tok, nxt.tolist() if kind is list else nxt.astype(kind), [0, 1, 0])
    assert tok.got == (nxt.tolist(), [0, 1, 0])


@pytest.mark.parametrize("bad", [2**32 + 1, 2**31, -2**31 - 1, -2**40, 0.5, float("nan")])
def test_next_states_that_32_bits_do_not_hold_are_refused(bad):
    nxt, tok = _next().astype(np.float64 if isinstance(bad, float) else np.int64), _Tok()
    nxt[1, 7] = bad
    with pytest.raises(ValueError):
        pkg.Grammar(tok, nxt, [0, 1, 0])
    assert tok.got is None


@pytest.mark.parametrize("accept", [[False, True, True], [0, 256, -1], [0.0, 0.5, 3.0], np.array([0, 1, 255], np.uint8)])
def test_accept_is_whether_a_value_is_not_0(accept):
    tok = _Tok()
    pkg.Grammar(tok, _next(), accept)
    assert tok.got[1] == [0, 1, 1]
