"""smoke() compares what it says it compares: a gradient of the norms that is off by a part in a thousand is noticed."""
import pytest

import hadamard_rotation_gb300 as hq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from hadamard_rotation_gb300 import build
    import oracle

    build.build()
    oracle.build()


def test_smoke():
    import __graft_entry__

    __graft_entry__.smoke()


@pytest.mark.parametrize("which", [0, 1, 3, 4])
def test_smoke_notices_a_wrong_gradient(monkeypatch, which):
    import __graft_entry__

    right = hq.hq_block_norm_bwd

    def wrong(*args, **kw):
        out = list(right(*args, **kw))
        out[which] = out[which] * 1.001
        return tuple(out)

    monkeypatch.setattr(hq, "hq_block_norm_bwd", wrong)
    with pytest.raises(AssertionError, match="norms' gradient"):
        __graft_entry__.smoke()
