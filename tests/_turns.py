"""The angles of rotary positions to 50 digits, without floating point."""
from decimal import Decimal, getcontext

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def exact_turns(rot, base, scaling="none", by=1.0, original=8192.0, low=1.0, high=32.0):
    """Turns per position of each pair, to 50 digits."""
    getcontext().prec = 60
    b, by = Decimal(base), Decimal(by)
    if scaling == "base":
        b *= by ** (Decimal(rot) / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = (b.ln() * (Decimal(-2 * i) / rot)).exp()
        if scaling == "linear":
            f /= by
        if scaling == "parts":
            g = min(Decimal(1), max(Decimal(0), (Decimal(original) * f / (2 * PI) - Decimal(low)) / Decimal(high - low)))
            f *= g + (1 - g) / by
        out.append(f / (2 * PI))
    return out


def exact_angles(turns, positions):
    """Radians of each position and pair, less whole turns."""
    return [[float(p * t % 1 * 2 * PI) for t in turns] for p in positions]
