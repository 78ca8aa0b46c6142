"""Plain forms of a paged cache's table operators (test infrastructure only), one row
after the other on the host, from the definitions in include/dcp_mla_pages.h."""
from __future__ import annotations


def share(n: int, cp: int, shard: int, interleave: int) -> int:
    """How many of the first n positions shard has."""
    return sum(p // interleave % cp == shard for p in range(max(n, 0))) if cp > 1 else max(n, 0)


def pages_of(row, P):
    """A row's pages: its entries before the first that is none."""
    out = []
    for e in row:
        if not 0 <= e < P:
            break
        out.append(e)
    return out


def update(tables, refs, parents, keeps, wants, page, cp=1, shard=0, interleave=1):
    """(tables, refs, copies, missing) as lists. tables: list of rows."""
    B, M, P = len(tables), len(tables[0]) if tables else 1, len(refs)
    refs = list(refs)
    old = [pages_of(r, P) for r in tables]
    new, plan = [], []
    for b in range(B):
        some = 0 <= parents[b] < B
        keep = min(share(keeps[b], cp, shard, interleave), M * page) if some else 0
        want = min(share(wants[b], cp, shard, interleave), M * page)
        new.append(old[parents[b]][:-(-keep // page)] if some else [])
        plan.append((keep, want))
    for b in range(B):
        for e in old[b]:
            refs[e] -= 1
        for e in new[b]:
            refs[e] += 1
    free = [e for e in range(P) if refs[e] == 0]
    about = {}  # page -> rows that are about to write behind kept tokens in it
    for b, (keep, want) in enumerate(plan):
        if want > keep and keep % page and keep // page < len(new[b]):
            about.setdefault(new[b][keep // page], []).append(b)
    holders = {e: refs[e] for e in about}
    copies, missing = [[-1, -1] for _ in range(B)], 0

    def fresh():
        nonlocal missing
        if not free:
            missing += 1
            return -1
        e = free.pop(0)
        refs[e] = 1
        return e

    for b, (keep, want) in enumerate(plan):
        i = keep // page
        e = new[b][i] if i < len(new[b]) else None
        if e in about and b in about[e] and (holders[e] > len(about[e]) or about[e][-1] != b):
            refs[e] -= 1
            new[b][i] = fresh()
            if new[b][i] >= 0:
                copies[b] = [e, new[b][i]]
        for _ in range(len(new[b]), max(-(-keep // page), -(-want // page))):
            new[b].append(fresh())
    return [r + [-1] * (M - len(r)) for r in new], refs, copies, missing


def compact(tables, refs):
    """(tables, refs, copies without the empty pairs)."""
    P, refs = len(refs), list(refs)
    n = sum(r > 0 for r in refs)
    moves = list(zip([e for e in range(n, P) if refs[e] > 0], [e for e in range(n) if refs[e] <= 0]))
    to = dict(moves)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    return [[to.get(e, e) for e in r] for r in tables], refs, [list(m) for m in moves]
