"""How a warp of pa_beam_select with up to 8 beams raises its threshold in a chunk of which too
many values reach it, replayed on the CPU: in every chunk, whatever of it is NaN, it comes to an
end, and the W best numbers are among the values that are left."""
import numpy as np
import pytest

LANES, EACH, MANY = 32, 16, 64
CHUNK = LANES * EACH
LOWEST = np.finfo(np.float32).min
TURNS = 8  # (a turn that changes nothing repeats for ever)


def ordered(x):
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return u ^ np.where(u >> 31, np.uint32(0xffffffff), np.uint32(0x80000000))


def unordered(o):
    return (o ^ np.where(o >> 31, np.uint32(0x80000000), np.uint32(0xffffffff))).view(np.float32)


def lanes(x, n):
    """Chunks [N, 512] by lanes: 16 bytes of n values each time, or (1) single values."""
    return x.reshape(-1, EACH // n, LANES, n).swapaxes(1, 2).reshape(-1, LANES, EACH)


def with_nan(x, mt, t, W):
    """The order of all lanes' maxima, and left where the W-th is not above t."""
    reached = np.sort(ordered(mt), 1)[:, LANES - W]
    return reached, unordered(reached) <= t


def of_numbers(x, mt, t, W):
    o = np.where(mt >= t[:, None], ordered(mt), np.uint32(0))
    reached = np.sort(o, 1)[:, LANES - W]
    return reached, ~(unordered(reached) > t)


def thresholds(x, t, W, turn):
    """Chunks by lanes and their thresholds before; those after, and turns."""
    x, t = x.copy(), t.astype(np.float32)
    mt = np.fmax.reduce(x, 2)  # (NaN of a lane of nothing else)
    going = (mt >= t[:, None]).any(1)
    reached = np.zeros(len(x), np.uint32)
    turns = np.zeros(len(x), int)
    for _ in range(TURNS):
        t = np.where(going, np.fmax(t, unordered(np.maximum(reached, ordered(LOWEST)))), t)
        going &= (x >= t[:, None, None]).sum((1, 2)) > MANY
        if not going.any():
            break
        turns += going
        now, last = turn(x, mt, t, W)
        reached = np.where(going, now, reached)
        going &= ~last
    return t, np.where(going, TURNS + 1, turns)


def patterns(rng):
    """Chunks [N, 512] with NaN at some places."""
    at = np.arange(CHUNK)
    nan = [at < n for n in range(CHUNK + 1)] + [at >= n for n in range(CHUNK)]
    nan += [at // 16 % 32 < n for n in range(33)] + [at % 32 < n for n in range(33)]
    nan += [at // 8 % 32 < n for n in range(33)] + [at // 4 % 32 < n for n in range(33)]
    nan += [rng.random(CHUNK) < share for share in np.linspace(0, 1, 21) for _ in range(40)]
    nan = np.array(nan)
    x = rng.standard_normal(nan.shape).astype(np.float32)
    steps = np.round(x).astype(np.float32)  # equal ones
    far = np.where(rng.random(nan.shape) < 0.1, rng.choice([-np.inf, np.inf], nan.shape), x)
    low = np.where(rng.random(nan.shape) < 0.5, -np.inf, x)
    return [np.where(nan, np.float32(np.nan), y).astype(np.float32) for y in (x, steps, far, low)]


@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("n", [1, 4, 8])  # odd rows; aligned ones of 32 bits, of 16
def test_every_chunk_ends(W, n):
    rng = np.random.default_rng(W + n)
    with np.errstate(invalid="ignore"):
        for x in patterns(rng):
            x = lanes(x, n)
            for before in (LOWEST, -0.5, 1.0):
                t0 = np.full(len(x), before, np.float32)
                t, turns = thresholds(x, t0, W, of_numbers)
                assert (turns <= 2).all()
                assert (t >= t0).all()
                # of what reached it before, the W best still do
                flat = x.reshape(len(x), -1)
                best = -np.sort(-np.where(flat >= t0[:, None], flat, -np.inf), 1)[:, :W]
                assert ((best >= t[:, None]) | (best == -np.inf)).all()


@pytest.mark.parametrize("W,n,first", [(1, 4, 400), (2, 4, 400), (4, 4, 400), (1, 8, 264),
                                       (4, 8, 288), (8, 8, 320)])
def test_an_order_with_nan_is_seen(W, n, first):
    """NaN in the order of the maxima is above all numbers and raises nothing."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, CHUNK)).astype(np.float32)
    x[:, :first] = np.nan
    t0 = np.full(1, LOWEST)
    with np.errstate(invalid="ignore"):
        assert thresholds(lanes(x, n), t0, W, with_nan)[1] > TURNS
        assert thresholds(lanes(x, n), t0, W, of_numbers)[1] <= 2
