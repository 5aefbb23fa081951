"""examples/serve_attention.py: the cache operators as one program."""
import importlib.util
import os

import pytest

from tests.gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_attention.py")
    spec = importlib.util.spec_from_file_location("serve_attention", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("hq,hkv,d,prefix,lengths", [(8, 2, 64, 70, [1, 33, 20]), (6, 1, 128, 129, [40, 1]),
                                                     (4, 4, 256, 16, [5])])
def test_steps_and_graph_agree(hq, hkv, d, prefix, lengths):
    """A graph of a step replays what single calls compute, and both are the
    plain attention over the rows read back."""
    torch = need_gpu()
    m = example()
    log(f"serving example {hq} heads of {d}, prefix {prefix}, prompts {lengths}")
    hidden, steps = 512, 4

    def server():
        return m.Server(2, hidden, hq, hkv, d, 32, len(lengths), prefix, max(lengths) + steps + 1)

    gen = torch.Generator(device="cuda").manual_seed(3)
    xp = torch.randn((prefix, hidden), generator=gen, device="cuda").bfloat16()
    xo = torch.randn((sum(lengths), hidden), generator=gen, device="cuda").bfloat16()
    ends = torch.tensor(lengths).cumsum(0).cuda() - 1
    s, g = server(), server()
    xs = []
    for srv in (s, g):
        srv.fill_prefix(xp, 64)
        xs.append(srv.fill_prompts(xo, lengths)[ends].contiguous())
    assert torch.equal(xs[0].view(torch.int16), xs[1].view(torch.int16))
    graph = m.captured(g, xs[1])
    for i in range(steps):
        kept = {}
        s.step(xs[0], kept)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(xs[0].view(torch.int16), xs[1].view(torch.int16)), f"step {i}"
        assert torch.equal(s.lens, g.lens)
        want = s.plain_attention(kept["q"], s.layers[-1])
        # the rows read back are rounded to bf16 (2^-9 of each key and value, so
        # of scores that are sums of D products of at most |q||k| scale), and
        # the output once more
        err = (kept["o"].float() - want).norm() / want.norm()
        assert err < 2.0 ** -6, f"step {i}: {err}"


def test_main_prints_a_rate(capsys):
    need_gpu()
    example().main(["--layers", "1", "--hidden", "512", "--q-heads", "4", "--kv-heads", "2", "--head-dim", "64", "--batch",
                    "3", "--prefix", "100", "--chunk", "64", "--prompt", "20", "--steps", "3", "--check"])
    out = capsys.readouterr().out
    assert "ms a step" in out and "relative error" in out


def test_main_without_a_prefix(capsys):
    need_gpu()
    log("serving example without a shared prefix")
    example().main(["--layers", "2", "--hidden", "512", "--q-heads", "4", "--kv-heads", "2", "--head-dim", "128", "--batch",
                    "1", "--prefix", "0", "--prompt", "20", "--steps", "3", "--check"])
    out = capsys.readouterr().out
    assert "ms a step" in out and "relative error" in out
