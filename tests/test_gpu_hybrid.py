"""The hybrid stack of gated-delta-rule and attention layers: prompts in one or several parts, single tokens, training."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_chunked_chunk_gb300 import build
    build.build()


def _stack(**kw):
    from gated_deltanet_chunked_chunk_gb300.hybrid import HybridStack
    return HybridStack(**kw)


def _prompts(lens, seed=3):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(n, 512, generator=gen).to("cuda", torch.bfloat16) for n in lens]


def _rms(x):
    return float(x.float().square().mean().sqrt())


def _run(stack, prompts, parts):
    """parts: for every step the new tokens of each request; returns every request's outputs."""
    at, out = [0] * len(prompts), [[] for _ in prompts]
    for news in parts:
        y = stack.step(torch.cat([p[a:a + m] for p, a, m in zip(prompts, at, news)]), list(news))
        for n, piece in enumerate(y.split(list(news))):
            out[n].append(piece)
        at = [a + m for a, m in zip(at, news)]
    return [torch.cat(o) for o in out]


def test_prompts_in_parts_and_token_by_token():
    """The same tokens in one step, in two and one by one.  Whole pages have the same codes either way, and sums differ
    in the last bits of bf16 (2^-8 a rounding, a handful in a row: 3 %); a page that fills token by token may round an
    8-bit code (2^-4 at most, about 2 % as a root mean square) more than once: 7 %."""
    lens = [192, 130, 67]
    prompts = _prompts(lens)
    whole = _stack(requests=3, context=256)
    a = _run(whole, prompts, [lens])
    assert int(whole.status) == 0 and whole.lens.tolist() == lens
    assert int(whole.num_free) == 3 * 4 - (3 + 3 + 2)
    again = _run(_stack(requests=3, context=256), prompts, [lens])
    two = _stack(requests=3, context=256)
    b = _run(two, prompts, [[128, 64, 64], [64, 66, 3]])
    assert int(two.status) == 0 and int(two.num_free) == int(whole.num_free)
    one = _stack(requests=3, context=256)
    c = _run(one, prompts, [[128, 66, 3]] + [[1, 1, 1]] * 64)
    assert int(one.status) == 0 and one.lens.tolist() == lens
    for x, y, z, r in zip(a, b, c, again):
        assert torch.equal(x, r)
        assert _rms(x.float() - y.float()) < 0.03 * _rms(x)
        assert _rms(x.float() - z.float()) < 0.07 * _rms(x)


def test_training_lowers_the_loss():
    x, t = _prompts([200, 200], seed=5)
    stack = _stack(requests=1)
    losses = [stack.train_step(x, t, 0.5) for _ in range(4)]
    assert all(l2 < l1 for l1, l2 in zip(losses, losses[1:])), losses


def test_command(capsys):
    from gated_deltanet_chunked_chunk_gb300 import hybrid
    hybrid.main(["--requests", "3", "--prompt", "70", "--tokens", "3"])
    assert "status 0" in capsys.readouterr().out
