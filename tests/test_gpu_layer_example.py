"""The example of a linear-attention layer runs, and its serving path gives what
the layer's definition gives in 64 bits from the same projections."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from examples.linear_attention_layer import Layer, main, serve
from tests import layer_reference as ref
from tests.gpu_util import TOL_BF16, ensure_lib, rel_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def test_example_runs(capsys):
    main()
    assert "served" in capsys.readouterr().out and binding.device_error() == 0


def test_serving_follows_the_recurrence(monkeypatch):
    """Every request's tokens in order through the token recurrence, the forked
    request's from its parent's state on."""
    seen = {}

    def spy(name):
        f = getattr(binding, name)

        def call(q, k, v, g, *args, **kw):
            got = f(q, k, v, g, *args, **kw)
            seen.setdefault(name, []).append((q.clone(), k.clone(), v.clone(), g.clone(), kw, got))
            return got
        monkeypatch.setattr(binding, name, call)

    spy("linattn_chunk_fwd")
    spy("linattn_step")
    lengths = (37, 130, 5)
    layer = Layer()
    _, requests, n_live = serve(layer, lengths)
    assert n_live == 3 and sorted(requests.tolist()) == [0, 1, 2]
    (q, k, v, g, _, (o, states)), = seen["linattn_chunk_fwd"]
    want, want_s = ref.linattn(q, k, v, g, None, list(lengths), layer.scale)
    assert rel_err(o, want) <= TOL_BF16 and rel_err(states, want_s) <= 1e-5
    state = torch.cat([want_s, want_s[1:2]])  # the fork
    for i, (q, k, v, g, kw, o) in enumerate(seen["linattn_step"]):
        if i == 3:
            state = state[1:]  # the first request has ended
        want, state = ref.step(q, k, v, g, state, None, None, layer.scale)
        # steps are exact but for o's rounding; the first state carries the prompt's 1e-5
        assert rel_err(o, want) <= TOL_BF16
