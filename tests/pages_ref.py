"""The page bookkeeping's definition in plain integers, one request at a time."""


def share(n, r, N):
    return n // N + (1 if r < n % N else 0)


def entries(n, r, N, page):
    return -(-share(n, r, N) // page)


def member(b, groups, N, page, max_len, max_pages):
    """(first request, common entries) of request b; groups = (group_start, prefix_lens) or None."""
    if groups is not None:
        gs, pl = groups
        for g in range(len(pl)):
            if gs[g] <= b < gs[g + 1] and gs[g] != b:
                return gs[g], min(min(max(pl[g], 0), max_len) // N // page, max_pages)
    return b, 0


def reserve(cached, new, max_len, T, num_pages, page, table, free, count, groups=None):
    """table [N][B][max_pages] and the rest as lists; what dcp_page_reserve writes, as a dict (rows behind the last
    token left out)."""
    N, B, mp = len(table), len(cached), len(table[0][0]) if table[0] else 0
    table = [[list(row) for row in rank] for rank in table]
    out = dict(query_start=[0], seq_lens=[], positions=[], slots=[], requests=[], missing=[0] * N, free_count=list(count))
    at = out["query_start"]
    for b in range(B):
        n = max(0, min(new[b], max_len - cached[b]))
        n = min(n, T - at[-1])
        at.append(at[-1] + n)
        out["seq_lens"].append(cached[b] + n)
        first, common = member(b, groups, N, page, max_len, mp)
        for r in range(N):
            for j in range(max(entries(cached[b], r, N, page), common), entries(cached[b] + n, r, N, page)):
                if out["free_count"][r] > 0:
                    out["free_count"][r] -= 1
                    table[r][b][j] = free[r][out["free_count"][r]]
                else:
                    out["missing"][r] += 1
                    table[r][b][j] = -1
            for j in range(common):
                table[r][b][j] = table[r][first][j]
        for g in range(cached[b], cached[b] + n):
            r, i = g % N, g // N
            pg = table[r][b][i // page]
            out["positions"].append(g)
            out["requests"].append(b)
            out["slots"].append((r * num_pages + pg) * page + i % page if 0 <= pg < num_pages else -1)
    out["block_table"] = table
    return out


def release(lens, keep, max_len, num_pages, page, table, free, count, groups=None):
    N, mp = len(table), len(table[0][0]) if table[0] else 0
    free, count, cap = [list(f) for f in free], list(count), len(free[0])
    kept = [l if k < 0 else min(k, l) for l, k in zip(lens, keep)]
    for r in range(N):
        for b, (l, k) in enumerate(zip(lens, kept)):
            _, common = member(b, groups, N, page, max_len, mp)
            for j in range(max(entries(k, r, N, page), common), entries(l, r, N, page)):
                if 0 <= table[r][b][j] < num_pages:
                    if count[r] < cap:
                        free[r][count[r]] = table[r][b][j]
                    count[r] += 1
        count[r] = min(count[r], cap)
    return dict(free_pages=free, free_count=count, lens_out=kept)
