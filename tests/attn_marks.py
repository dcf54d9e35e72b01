"""Values that show every part of a long cache in the output: V is 0 but at marked tokens, where it is 1 in the dim of the
token's block, so a dim of the output is the weight of a few blocks' marked tokens.  A block, or one token of it, that is
left out or taken twice moves that dim by a part of it that is far more than the roundings."""
import torch

EPS16 = 2.0 ** -8


def blocks(n, step, D, at=None):
    """V [n, D]: token i's mark is in dim (i // step) % D; with `at`, only tokens at that place of their block have one."""
    i = torch.arange(n)
    v = torch.zeros(n, D)
    marked = i if at is None else i[i % step == at]
    v[marked, (marked // step) % D] = 1.0
    return v


def equal_weights(v):
    """What attention with equal scores gives: the mean, exact to the roundings below."""
    return v.double().mean(0)


def close(got, want):
    """Equal weights and their products are powers of two times whole numbers below 2^24: the sums are exact, and left are
    the quotient's rounding in fp32 and the output's to bf16."""
    return (got.double() - want).abs() <= want * (EPS16 + 3 * 2.0 ** -24)


def cache_of(vs, page, kind, scale=0.5, seed=0):
    """(k, v pages, table) on the host of sequences that share one kv head count: vs of [n, Hkv, D] each, K random, pages
    shuffled; for e4m3 values are stored divided by scale."""
    g = torch.Generator().manual_seed(seed)
    Hkv, D = vs[0].shape[1:]
    counts = [-(-v.shape[0] // page) for v in vs]
    order = torch.randperm(sum(counts) + 1, generator=g)
    v_pages = torch.zeros(len(order), Hkv, page, D)
    table = torch.full((len(vs), max(1, max(counts))), -1, dtype=torch.int32)
    for b, (v, count) in enumerate(zip(vs, counts)):
        mine, order = order[:count], order[count:]
        table[b, :count] = mine.int()
        held = torch.zeros(count * page, Hkv, D)
        held[: v.shape[0]] = v
        v_pages[mine] = held.view(count, page, Hkv, D).transpose(1, 2)
    k_pages = torch.randn(v_pages.shape, generator=g)
    if kind == "e4m3":
        return (k_pages.to(torch.float8_e4m3fn), (v_pages / scale).to(torch.float8_e4m3fn)), table
    return (k_pages.to(torch.bfloat16), v_pages.to(torch.bfloat16)), table
