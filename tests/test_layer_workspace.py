"""Workspaces of the training and serving calls: the query grows with the number of tokens and the rank, so that the
workspace of the longest prompt serves every shorter one."""
import pytest
import torch

QUERIES = ["qlora_forward_dropout_workspace_bytes", "qlora_backward_workspace_bytes",
           "mxfp4_forward_workspace_bytes", "mxfp4_backward_workspace_bytes"]


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("rows,cols", [(4096, 4096), (11008, 4096), (4096, 11008), (28672, 8192), (130, 64), (64, 16384),
                                       (5, 640)])
def test_query_grows_with_the_tokens_and_the_rank(query, rows, cols):
    from loftq_qlora_initialization_amd import binding as b
    q = getattr(b, query)
    counts = list(range(0, 4200)) + [int(1.3 ** k) for k in range(33, 50)]
    before = None
    for r in (0, 1, 16, 17, 33, 64):
        need = [q(n, rows, cols, r) for n in counts]
        assert need == sorted(need)
        assert before is None or all(x <= y for x, y in zip(before, need))
        before = need


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
def test_one_workspace_for_every_prompt(lib, mx):
    """Counts at which K ranges begin and end, from the longest to one token, in its workspace filled with NaN: results
    as with a workspace of their own, and nothing written behind it."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, cols, r, longest = 1040, 2048, 16, 2300

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    X, G = normal(longest, cols, dtype=torch.bfloat16), normal(longest, rows, dtype=torch.bfloat16)
    W, ad = normal(rows, cols), dict(B=normal(rows, r), A=normal(r, cols))
    if mx:
        base = dict(zip(("packed", "scales"), lib.loftq_mxfp4_quantize(W)))
        fwd, bwd = lib.loftq_mxfp4_forward, lib.loftq_mxfp4_backward
        qf, qb = lib.mxfp4_forward_workspace_bytes, lib.mxfp4_backward_workspace_bytes
    else:
        base = dict(zip(("packed", "absmax"), lib.loftq_nf4_quantize(W)))
        fwd, bwd = lib.loftq_qlora_forward_dropout, lib.loftq_qlora_backward
        qf, qb = lib.qlora_forward_dropout_workspace_bytes, lib.qlora_backward_workspace_bytes
    wf, wb = (torch.full((q(longest, rows, cols, 64) + 4096,), 255, dtype=torch.uint8, device="cuda") for q in (qf, qb))
    for n in (2300, 2049, 1100, 1025, 700, 513, 384, 257, 129, 128, 77, 65, 33, 17, 16, 9, 8, 1):
        for adapter in (ad, {}):
            kw = dict(shape=(rows, cols), **base, **adapter)
            own = dict(f=qf(n, rows, cols, r if adapter else 0), b=qb(n, rows, cols, r if adapter else 0))
            small = {k: torch.zeros(max(v, 16), dtype=torch.uint8, device="cuda") for k, v in own.items()}
            for p in ((0.0, 0.2) if adapter else (0.0,)):
                rng = dict(p=p, seed=3, offset=n)
                got = fwd(X[:n], ws=wf[:-4096], **kw, **rng), *bwd(G[:n], X[:n], ws=wb[:-4096], **kw, **rng)
                want = fwd(X[:n], ws=small["f"], **kw, **rng), *bwd(G[:n], X[:n], ws=small["b"], **kw, **rng)
                for a, c in zip(got, want):
                    assert (a is None and c is None) or torch.equal(a, c), n
    assert (wf[-4096:] == 255).all() and (wb[-4096:] == 255).all()
