"""What atlas.cross refuses before anything is launched: tensors of the wrong shape, type,
device or layout, each one away from a call that it answers."""
import pytest
import torch

import exact_causal_gqa_gb300 as atlas

B, HQ, HKV, N, D, P, PAGES, WIDTH = 3, 8, 2, 5, 64, 16, 12, 4


def call(device, **change):
    """The arguments of a good call with some of them replaced; `change` maps a name to a
    tensor, a number, or a function of what stands there."""
    bf16, i32 = dict(dtype=torch.bfloat16, device=device), dict(dtype=torch.int32, device=device)
    x = dict(q=torch.ones((B, HQ, N, D), **bf16), k_pages=torch.ones((PAGES, HKV, P, D), **bf16),
             v_pages=torch.ones((PAGES, HKV, P, D), **bf16), page_table=torch.arange(B * WIDTH, **i32).reshape(B, WIDTH),
             enc_lens=torch.tensor([60, 0, 7], **i32), n_q_heads=HQ, n_kv_heads=HKV, head_dim=D,
             page_tokens=P, scale=0.1, out=torch.zeros((B, HQ, N, D), **bf16),
             lse=torch.zeros((B, HQ, N), device=device), status=torch.zeros(1, **i32),
             sinks=torch.zeros(HQ, device=device), q_lens=torch.tensor([5, 1, 0], **i32))
    for name, to in change.items():
        x[name] = to(x.get(name)) if callable(to) else to
    return x


def test_tensors_on_the_host():
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        atlas.cross(**call("cpu"))


def apart(t):
    """The same shape and values, not contiguous."""
    return torch.stack([t, t], -1)[..., 0]


BAD = [
    ("q", lambda t: t[0]), ("q", lambda t: t[:, :4].contiguous()), ("q", lambda t: t[..., :32].contiguous()),
    ("q", lambda t: t[:2]), ("q", apart), ("q", lambda t: t.float()),
    ("k_pages", lambda t: t[:, :1].contiguous()), ("k_pages", lambda t: t[:, :, :8].contiguous()),
    ("k_pages", lambda t: t[0]), ("k_pages", lambda t: t.float()), ("k_pages", apart), ("k_pages", lambda t: t.cpu()),
    ("v_pages", lambda t: t[:6]), ("v_pages", lambda t: t.float()), ("v_pages", apart), ("v_pages", lambda t: t.cpu()),
    ("page_table", lambda t: t[:2]), ("page_table", lambda t: t[0]), ("page_table", lambda t: t.long()),
    ("page_table", lambda t: t.t().contiguous()), ("page_table", apart), ("page_table", lambda t: t.cpu()),
    ("enc_lens", lambda t: t[:2]), ("enc_lens", lambda t: t.long()), ("enc_lens", apart), ("enc_lens", lambda t: t.cpu()),
    ("out", lambda t: t[:, :, :4].contiguous()), ("out", apart), ("out", lambda t: t.transpose(1, 2)),
    ("out", lambda t: t.cpu()), ("out_dtype", torch.float32),       # a bf16 out with room for half of it
    ("lse", lambda t: t.bfloat16()), ("lse", lambda t: t[:, :, :4].contiguous()), ("lse", apart), ("lse", lambda t: t.cpu()),
    ("status", lambda t: t.long()), ("status", lambda t: t[:0]), ("status", lambda t: t.cpu()),
    ("sinks", lambda t: t[:2]), ("sinks", lambda t: t.double()), ("sinks", apart), ("sinks", lambda t: t.cpu()),
    ("q_lens", lambda t: t[:2]), ("q_lens", lambda t: t.long()), ("q_lens", apart), ("q_lens", lambda t: t.cpu()),
    ("workspace", lambda t: torch.zeros((1 << 20, 2), dtype=torch.uint8, device="cuda")[:, 0]),
    ("workspace", lambda t: torch.zeros(1 << 20, dtype=torch.uint8)),
    ("n_q_heads", 4), ("n_kv_heads", 1), ("n_kv_heads", 4), ("head_dim", 128), ("page_tokens", 8),
]


@pytest.mark.gpu
@pytest.mark.parametrize("k", range(len(BAD)), ids=[f"{n}{i}" for i, (n, _) in enumerate(BAD)])
def test_one_wrong_tensor_or_size(k):
    x = call("cuda", **dict([BAD[k]]))
    with pytest.raises(ValueError):
        atlas.cross(**x)
    torch.cuda.synchronize()
    if BAD[k][0] not in ("out", "lse"):
        assert (x["out"] == 0).all() and (x["lse"] == 0).all()


@pytest.mark.gpu
def test_the_call_they_differ_from():
    """Every value row is 1: rows over states are L / (L + e^0 / e^s), rows over none 0."""
    x = call("cuda")
    assert atlas.cross(**x) is x["out"] and int(x["status"].item()) == 0
    # scores 64 * 0.1 each: L e^6.4 / (L e^6.4 + 1), rounded to bf16
    want = 60 * 2.718281828459045 ** 6.4
    assert (x["out"][0].float() - want / (want + 1)).abs().max() <= 2e-3 + 2.0 ** -8
    assert (x["out"][1:] == 0).all()                       # no states; q_lens[2] is 0: not written
    for change in (dict(out=None), dict(out=None, out_dtype=torch.float32), dict(lse=None, status=None),
                   dict(lse=lambda t: t.reshape(-1)), dict(sinks=None, q_lens=None),
                   dict(out=lambda t: t.float(), out_dtype=torch.float32),
                   dict(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))):
        y = call("cuda", **change)
        out = atlas.cross(**y)
        assert out.dtype == (y.get("out_dtype") or torch.bfloat16) and out.shape == x["out"].shape
        if y["sinks"] is not None:
            assert torch.equal(out[0].to(torch.bfloat16), x["out"][0])


@pytest.mark.gpu
def test_the_library_refuses_what_has_no_meaning_here():
    for kw in (dict(window=4), dict(phase=1), dict(chunk_range=torch.zeros((B, 2), dtype=torch.int32, device="cuda"))):
        with pytest.raises(atlas.AtlasError):
            atlas.cross(**call("cuda"), **kw)
    with pytest.raises(TypeError):
        atlas.cross(**call("cuda"), windows=4)


@pytest.mark.gpu
def test_from_host_tensors_the_same_is_refused():
    x = call("cpu")
    args = [x[n] for n in ("q", "k_pages", "v_pages", "page_table", "enc_lens")]
    sizes = HQ, HKV, D, P, 0.1
    got = atlas.run_host("cross", *args, *sizes)
    assert torch.equal(got, atlas.cross(*(t.cuda() for t in args), *sizes).cpu())
    for k, bad in ((3, args[3][:2]), (4, args[4][:2]), (2, args[2].float()), (1, args[1][:, :1])):
        with pytest.raises(ValueError):
            atlas.run_host("cross", *args[:k], bad, *args[k + 1:], *sizes)
