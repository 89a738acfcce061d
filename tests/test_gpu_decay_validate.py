"""LA_VALIDATE=1 looks at every decay, however many heads there are."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


@pytest.mark.parametrize("H", [1, 255, 256, 257, 1000])
def test_every_head(la, monkeypatch, H):
    monkeypatch.setenv("LA_VALIDATE", "1")
    x = torch.zeros(1, H, 64, device="cuda")
    S = torch.zeros(1, H, 64, 64, device="cuda")
    g = torch.full((H,), -0.5, device="cuda")
    la.decode_step(x, x, x, S, log_decay=g)
    for h in {0, H // 2, H - 1}:
        bad = g.clone()
        bad[h] = 0.25
        with pytest.raises(la.LAError, match=rf"log_decay\[{h}\]"):
            la.decode_step(x, x, x, S, log_decay=bad)
