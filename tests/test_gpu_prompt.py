"""A whole text prompt over the handle's detailed state D: rotation at the
virtual positions, rows appended to D, attention over all earlier rows and,
causally, the prompt's own.  Tolerances as in test_gpu_text_handle.py."""

import pytest
import torch

import kv_cache_compression_frame_gb300 as kv
from test_gpu_text_handle import _built, check_attention, check_rotated, handle, rows_of, text  # noqa: F401
from test_text_ops import DEV, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,norm,heads", [(128, False, (6, 2)), (64, True, (14, 2)), (128, False, (16, 1))])
def test_prompt_over_the_detailed_state(d, norm, heads):
    h = handle(head_dim=d, num_q_heads=heads[0], num_kv_heads=heads[1])
    c, g = h.cfg, gen(d)
    qw = kw = None
    if norm:
        qw, kw = (1 + randn(g, c.num_layers, d, dtype=torch.float32) / 4 for _ in range(2))
        h.set_qk_norm(qw, kw)
    for _ in range(3):
        h.prefill_frame(*text(h, g, c.frame_tokens))
    first = 3 * c.frame_tokens
    for tok in (1, 37, 64, 2):
        q, k, v = text(h, g, tok)
        dk, dv = rows_of(h, "k"), rows_of(h, "v")
        o = h.decode_prompt(q, k, v)
        h.check_device_status()
        pos = (c.position_offset + first + torch.arange(tok, device=DEV)).expand(c.num_streams, tok)
        qr = h.rotated_query().reshape(-1)[:q.numel()].view(q.shape).clone()
        check_rotated(qr, q, pos, h.omega64, qw, 1e-6)
        nk, nv = rows_of(h, "k"), rows_of(h, "v")
        check_rotated(nk[..., first:first + tok, :], k, pos, h.omega64, kw, 1e-6)
        assert torch.equal(nv[..., first:first + tok, :], v)
        mask = torch.ones(tok, first + tok, dtype=torch.bool, device=DEV).tril(first).expand(c.num_streams, -1, -1)
        check_attention(h, qr, nk[..., :first + tok, :], nv[..., :first + tok, :], mask, o)
        nk[..., first:first + tok, :], nv[..., first:first + tok, :] = \
            dk[..., first:first + tok, :], dv[..., first:first + tok, :]
        assert torch.equal(nk, dk) and torch.equal(nv, dv)
        first += tok
    assert h.text_tokens == 104 and h.detailed(0, 0)[2] == first


def test_prompt_then_tokens_is_one_text():
    """A prompt, then decode(): the same rows of D as decode() alone in fours."""
    a, b, g = handle(), handle(), gen(9)
    for _ in range(2):
        x = text(a, g, a.cfg.frame_tokens)
        a.prefill_frame(*x)
        b.prefill_frame(*x)
    q, k, v = text(a, g, 16)
    a.decode_prompt(*(x[..., :12, :].contiguous() for x in (q, k, v)))
    a.decode(*(x[..., 12:, :].contiguous() for x in (q, k, v)))
    for i in range(0, 16, 4):
        b.decode(*(x[..., i:i + 4, :].contiguous() for x in (q, k, v)))
    assert a.text_tokens == b.text_tokens == 16
    assert torch.equal(rows_of(a, "k"), rows_of(b, "k")) and torch.equal(rows_of(a, "v"), rows_of(b, "v"))


def test_prompt_captured_and_on_another_stream():
    h, g = handle(), gen(10)
    h.prefill_frame(*text(h, g, 64))
    x = text(h, g, 20)
    h.decode_prompt(*x)                               # allocates
    want = h.decode_prompt(*x)
    h.reset()
    h.prefill_frame(*text(h, gen(10), 64))
    h.decode_prompt(*x)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        h.decode_prompt(*x, o=out)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h.decode_prompt(*x, stream=s)
    s.synchronize()
    h.check_device_status()


def test_prompt_on_another_stream_is_the_same():
    """Outputs, queries and appended rows, behind work of that stream that the
    default stream has not waited for."""
    g = gen(12)
    frames = [text(handle(), g, 64) for _ in range(2)]
    x = text(handle(), g, 30)
    got = []
    for s in (None, torch.cuda.Stream()):
        h = handle()
        for f in frames:
            h.prefill_frame(*f)
        h.decode_prompt(*(y[..., :7, :].contiguous() for y in x))                # allocates
        rest = [y[..., 7:, :].contiguous() for y in x]
        late = [torch.zeros_like(y) for y in rest]
        torch.cuda.synchronize()
        with torch.cuda.stream(s or torch.cuda.current_stream()):
            torch.cuda._sleep(20_000_000)
            for a, b in zip(late, rest):
                a.copy_(b)
        o = h.decode_prompt(*late, stream=s)
        torch.cuda.synchronize()
        h.check_device_status()
        got.append((o, h.rotated_query().reshape(-1)[:late[0].numel()].clone(), rows_of(h, "k")[..., :158, :],
                    rows_of(h, "v")[..., :158, :]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0].any()


def test_prompt_rules():
    h = handle(max_frames=2)
    g = gen(11)
    with pytest.raises(kv.StateKVError) as e:
        h.decode_prompt(*text(h, g, 65))              # more than a frame's tokens
    assert e.value.status == -1
    h.decode_prompt(*text(h, g, 64))                  # before any frame
    with pytest.raises(kv.StateKVError) as e:
        h.prefill_frame(*text(h, g, 64))              # text has begun
    assert e.value.status == -1
    h.decode_prompt(*text(h, g, 60))
    with pytest.raises(kv.StateKVError) as e:
        h.decode_prompt(*text(h, g, 5))               # D is full
    assert e.value.status == -3
    h.decode_prompt(*text(h, g, 4))
    h.check_device_status()
    f = handle(dtype="f32")
    with pytest.raises(kv.StateKVError) as e:
        f.decode_prompt(*text(f, g, 3))
    assert e.value.status == -2
