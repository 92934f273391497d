"""The ring of the routed layer's kernel, on the CPU: barriers that are waited for by the parity of a use, one
producing thread, several loading warps that take units in turn, one multiplying thread, in random order.  No place
is written before its last use is over as long as there are no more loading warps than places."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):  # the use of this parity is over
        return (self.phase & 1) != parity


def run(places, loaders, units, seed):
    """None, or what went wrong."""
    r = random.Random(seed)
    full, empty = [Barrier(2) for _ in range(places)], [Barrier(1) for _ in range(places)]
    weights, tokens = [None] * places, [None] * places
    issued, multiplied, next_of, flying = 0, 0, list(range(loaders)), []
    for _ in range(200000):
        if multiplied == units:
            return None
        who = r.choice(["produce", "land", "multiply", "load", "load", "load"])
        if who == "produce" and issued < units:
            s = issued % places
            if empty[s].done((issued // places & 1) ^ 1):
                flying.append((s, issued))
                issued += 1
        elif who == "land" and flying:
            s, u = flying.pop(r.randrange(len(flying)))
            if weights[s] is not None:
                return f"weights of unit {weights[s]} overwritten"
            weights[s] = u
            full[s].arrive()
        elif who == "load":
            w = r.randrange(loaders)
            u = next_of[w]
            if u < units and empty[u % places].done((u // places & 1) ^ 1):
                if tokens[u % places] is not None:
                    return f"tokens of unit {tokens[u % places]} overwritten"
                tokens[u % places] = u
                full[u % places].arrive()
                next_of[w] += loaders
        elif who == "multiply":
            s = multiplied % places
            if full[s].done(multiplied // places & 1):
                if (weights[s], tokens[s]) != (multiplied, multiplied):
                    return f"unit {multiplied} multiplied with {weights[s]} and {tokens[s]}"
                weights[s] = tokens[s] = None
                empty[s].arrive()
                multiplied += 1
    return "no end"


@pytest.mark.parametrize("places", [3, 4, 5, 6, 8, 12])
def test_as_many_loading_warps_as_places(places):
    assert all(run(places, min(8, places), 40, seed) is None for seed in range(40))


def test_more_loading_warps_than_places_go_wrong():
    assert any(run(5, 8, 40, seed) is not None for seed in range(40))
